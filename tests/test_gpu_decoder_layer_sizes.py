"""The example decoder layer at sizes that its products do not take as they are: experts that do not fill a tile of
16 weight rows, heads whose outputs do not fill a block of 128.

Tolerances as in test_gpu_decoder_layer: a request's first token attends to itself, so its attention output is its
value from the cache, off by 2^-4 of itself and 2^-10 of the page's largest; bf16 products and sums add 2^-6 of the row's
largest element.  Router logits: 2 (K + 8) 2^-24 of the sum of the products' magnitudes."""
import pytest
import torch

from harness import DEV, rdg
from test_gpu_decoder_layer import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_experts,n_q,n_kv,head_dim", [(8, 16, 4, 64), (4, 3, 1, 64), (12, 8, 2, 64), (20, 1, 1, 64), (40, 5, 5, 128)])
def test_layer_of_sizes_between_tiles(n_experts, n_q, n_kv, head_dim):
    m = rdg()
    layer = example().DecoderLayer(n_experts=n_experts, n_q=n_q, n_kv=n_kv, head_dim=head_dim, top_k=min(4, n_experts // 2), max_requests=3)
    g = torch.Generator(device=DEV).manual_seed(n_experts)
    x = torch.randn(3, layer.H, device=DEV, generator=g).bfloat16()
    layer.plan([1, 1, 1])
    got = layer.attention(x, 1).double()
    n = layer.norm(x).double()
    v = (n @ layer.w_qkv.double().T).view(3, -1, head_dim)[:, n_q + n_kv:].repeat_interleave(n_q // n_kv, 1).reshape(3, -1)
    w_o = layer.w_o.double()
    want = x.double() + v @ w_o.T
    bound = (2.0 ** -4 * v.abs() + 2.0 ** -10 * v.abs().max()) @ w_o.abs().T + 2.0 ** -6 * want.abs().max()
    assert ((got - want).abs() <= bound).all()

    router = layer.router.double()
    logits = layer.logits(layer.norm(x)).double()
    assert logits.shape == (3, n_experts)
    assert ((logits - n @ router.T).abs() <= 2 * (layer.H + 8) * 2.0 ** -24 * (n.abs() @ router.abs().T)).all()

    layer.keep([0, 0, 0])
    for q_len in ([9, 0, 30], [1, 4, 1], [1, 1, 1]):
        y = layer.forward(torch.randn(sum(q_len), layer.H, device=DEV, generator=g).bfloat16(), q_len)
        assert m.rdg_check_status(layer.step) == (0, 0) and torch.isfinite(y).all()
