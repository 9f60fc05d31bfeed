"""One decoder layer served with the library: attention over the paged 8-bit
cache, then the mixture-of-experts half, for prefill and decode steps.

    python examples/decoder_layer.py            (on an MI355X)

Random weights.  Requests arrive, are prefilled together, decode one token a
step beside newly arriving ones, and hand their pages back when they finish.
PyTorch supplies memory and streams; every step of the layer is the library's.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routing_dispatch_grouped_amd as rdg  # noqa: E402


class DecoderLayer:
    def __init__(self, hidden=512, n_q=16, n_kv=4, head_dim=64, n_experts=16, inner=256, top_k=4, page_rows=16,
                 n_pages=64, max_requests=8, max_context=256, max_tokens=256, device="cuda", seed=0,
                 score=rdg.RDG_SCORE_SIGMOID):
        g = torch.Generator(device=device).manual_seed(seed)
        self.H, self.n_q, self.n_kv, self.D = hidden, n_q, n_kv, head_dim
        self.N, self.I, self.K, self.dev = n_experts, inner, top_k, device
        self.max_context, self.n_pages, self.score = max_context, n_pages, score

        def weight(*shape):
            return (torch.randn(*shape, device=device, generator=g) * shape[-1] ** -0.5).bfloat16()

        self.w_qkv = weight((n_q + 2 * n_kv) * head_dim, hidden)
        self.w_o = weight(hidden, n_q * head_dim)
        self.gain_q = 1 + 0.1 * torch.randn(head_dim, device=device, generator=g)
        self.gain_k = 1 + 0.1 * torch.randn(head_dim, device=device, generator=g)
        self.router = weight(n_experts, hidden)

        def packed(w):
            if w.dim() == 2:  # products take rows by sixteens and columns by blocks of 128: zeros fill them up
                w = torch.nn.functional.pad(w, (0, -w.shape[1] % 128, 0, -w.shape[0] % 16))
            p = torch.empty_like(w)
            rdg.rdg_pack_weights(w, rdg.RDG_BF16, p)
            return p

        self.p_qkv, self.p_o, self.p_router = packed(self.w_qkv), packed(self.w_o), packed(self.router)
        self.w1, self.w3 = packed(weight(n_experts, inner, hidden)), packed(weight(n_experts, inner, hidden))
        self.w2 = packed(weight(n_experts, hidden, inner))
        # one workspace for the three products, of up to max_tokens
        self.work = torch.empty(max(rdg.rdg_linear_workspace_bound(max_tokens, *w.shape, rdg.RDG_BF16)
                                    for w in (self.p_qkv, self.p_o, self.p_router)), dtype=torch.uint8, device=device)
        angle = torch.arange(max_context, device=device)[:, None] * 10000.0 ** (
            -torch.arange(0, head_dim, 2, device=device) / head_dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        # the cache, its free pages, and the requests' rows
        self.cache = rdg.KvCache.empty(n_pages, n_kv, page_rows, head_dim, device)
        self.free = torch.arange(n_pages, dtype=torch.int32, device=device)
        self.n_free = torch.full((1,), n_pages, dtype=torch.int32, device=device)
        self.step = rdg.KvStep(max_requests, -(-max_context // page_rows), page_rows, n_pages, max_tokens, device)

    def plan(self, q_len):
        """q_len [max_requests]: new tokens of each request's row (0: none)."""
        q = torch.as_tensor(q_len, dtype=torch.int32, device=self.dev)
        rdg.rdg_kv_plan(self.step, self.step.kv_len, q, self.free, self.n_free, self.n_free)

    def keep(self, length):
        """length [max_requests]: tokens that each row keeps (0: finished)."""
        n = torch.as_tensor(length, dtype=torch.int32, device=self.dev)
        rdg.rdg_kv_trim(self.step, self.step.kv_len, n, self.free, self.n_free, self.n_free)

    @staticmethod
    def norm(x):
        out = torch.empty_like(x)
        rdg.rdg_add_norm(x, None, 1e-6, out=out)
        return out

    def linear(self, x, w, dtype=torch.bfloat16, residual=None):
        """x @ W.T (+ residual), W packed"""
        if x.shape[1] < w.shape[1]:
            x = torch.nn.functional.pad(x, (0, w.shape[1] - x.shape[1]))
        out = torch.empty(x.shape[0], w.shape[0], dtype=dtype, device=x.device)
        rdg.rdg_linear(x, None, rdg.RDG_BF16, w, None, out, residual=residual, work=self.work)
        return out

    def attention(self, x, max_q):
        T, n_q, D = x.shape[0], self.n_q, self.D
        qkv = self.linear(self.norm(x), self.p_qkv)
        q = torch.empty(T, n_q, D, dtype=x.dtype, device=self.dev)
        rdg.rdg_qk_norm_rope_store(qkv, n_q, self.n_kv, D, self.gain_q, self.gain_k, 1e-6, self.cos_sin, D, False, self.step,
                                   self.cache, q)
        out = torch.empty_like(q)
        work = torch.empty(rdg.rdg_paged_attention_workspace_bytes(self.cache, T, self.step.n_req, n_q, max_q,
                                                                   self.max_context, rdg.RDG_BF16),
                           dtype=torch.uint8, device=self.dev)
        rdg.rdg_paged_attention(q, self.step, self.cache, max_q, self.max_context, D ** -0.5, out, work=work)
        return self.linear(out.view(T, -1), self.p_o, residual=x)

    def logits(self, n):
        """The router's, of the experts that there are: rows may be apart."""
        return self.linear(n, self.p_router, torch.float32)[:, :self.N]

    def experts(self, x):
        T, H, K = x.shape[0], self.H, self.K
        n = self.norm(x)
        ids = torch.empty(T, K, dtype=torch.int32, device=self.dev)
        w = torch.empty(T, K, dtype=torch.float32, device=self.dev)
        rdg.rdg_route_topk(self.logits(n), self.score, 4, 2, 2, K, True, 1.0, ids, w)
        L = rdg.Layout(rdg.RDG_CONTIGUOUS, self.N, T, K, self.dev, block_m=16)
        rdg.rdg_dispatch(n, None, rdg.RDG_BF16, ids, L, None)
        h = torch.empty(L.m_cap, self.I, dtype=x.dtype, device=self.dev)
        y = torch.empty(L.m_cap, H, dtype=x.dtype, device=self.dev)
        rdg.rdg_grouped_ffn_gather(L, rdg.RDG_BF16, H, self.I, n, None, K, self.w1, self.w3, self.w2, None, None, None, h,
                                   None, y)
        out = torch.empty_like(x)
        rdg.rdg_combine(y, rdg.RDG_BF16, L, w, T, K, H, x, out, rdg.RDG_BF16)
        assert rdg.rdg_check_status(L) == (rdg.RDG_OK, 0)
        return out

    def forward(self, x, q_len):
        """x [sum(q_len), hidden] bf16: the step's tokens, row after row."""
        self.plan(q_len)
        return self.experts(self.attention(x, max(q_len)))


def main():
    torch.manual_seed(0)
    layer = DecoderLayer()
    waiting, done, lens, goal = [40, 5, 17, 33, 64, 1, 90, 12, 25, 70], 0, [0] * 8, [0] * 8
    steps = 0
    while waiting or any(lens):
        q_len = [1 if n else 0 for n in lens]
        for r in range(8):
            if lens[r] == 0 and waiting and sum(q_len) + waiting[0] <= 200:
                q_len[r] = waiting.pop(0)
                goal[r] = q_len[r] + 20
        x = torch.randn(sum(q_len), layer.H, device="cuda").bfloat16()
        y = layer.forward(x, q_len)
        assert rdg.rdg_check_status(layer.step) == (rdg.RDG_OK, 0) and torch.isfinite(y).all()
        lens = [n + q for n, q in zip(lens, q_len)]
        finished = [r for r in range(8) if lens[r] and lens[r] >= goal[r]]
        if finished:
            lens = [0 if r in finished else n for r, n in enumerate(lens)]
            done += len(finished)
            layer.keep(lens)
        steps += 1
    assert int(layer.n_free) == layer.n_pages
    print("decoder layer: %d requests served in %d steps, every page back" % (done, steps))


if __name__ == "__main__":
    main()
