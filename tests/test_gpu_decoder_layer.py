"""The example decoder layer: requests prefilled, decoded and released through
the whole path.  Its attention half is compared with a plain float64 layer that
keeps exact keys and values.

Tolerance: a cached value is off by at most half an e4m3 step, 2^-4 of itself
(2^-10 of its page's scale for the smallest), so a row's attention output is off by at most
2^-4 sum_j p_j |v_j| from the values and, the logits being off by at most e = 2^-4 scale
sum_d |q_d k_jd|, by a factor of up to exp(2 e) in each p_j.  These bounds are
several times the typical error; bf16 products and sums add 2^-6 of the row's largest element."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from harness import DEV, rdg
from oracle import paged

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_serves_its_requests():
    example().main()


def test_attention_half_against_exact_keys_and_values():
    m = rdg()
    layer = example().DecoderLayer(max_requests=3, seed=3)
    n_q, n_kv, D, scale = layer.n_q, layer.n_kv, layer.D, layer.D ** -0.5
    f64 = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    w_qkv, w_o, gq, gk, cs = (f64(t) for t in (layer.w_qkv, layer.w_o, layer.gain_q, layer.gain_k, layer.cos_sin))
    ks, vs = [[] for _ in range(3)], [[] for _ in range(3)]
    gen = torch.Generator(device=DEV).manual_seed(5)
    for q_len in ([5, 40, 0], [1, 1, 17], [1, 1, 1], [3, 0, 1], [1, 30, 1]):
        x = torch.randn(sum(q_len), layer.H, device=DEV, generator=gen).bfloat16()
        layer.plan(q_len)
        got = f64(layer.attention(x, max(q_len)))
        assert m.rdg_check_status(layer.step) == (0, 0)
        qkv = (f64(layer.norm(x)) @ w_qkv.T).reshape(-1, n_q + 2 * n_kv, D)
        t = 0
        for r, n in enumerate(q_len):
            for _ in range(n):
                pos = len(ks[r])
                c, s = cs[pos, :D // 2], cs[pos, D // 2:]
                q = paged.rotate(paged.norm(qkv[t, :n_q], gq, 1e-6), c, s, False)
                ks[r].append(paged.rotate(paged.norm(qkv[t, n_q:n_q + n_kv], gk, 1e-6), c, s, False))
                vs[r].append(qkv[t, n_q + n_kv:])
                K, V = np.stack(ks[r]), np.stack(vs[r])
                o, tol = np.zeros((n_q, D)), np.zeros((n_q, D))
                for h in range(n_q):
                    k, v = K[:, h * n_kv // n_q], V[:, h * n_kv // n_q]
                    logit = scale * k @ q[h]
                    p = np.exp(logit - logit.max())
                    p /= p.sum()
                    o[h] = p @ v
                    e = 2.0 ** -4 * scale * (np.abs(k) @ np.abs(q[h])).max()
                    tol[h] = (2.0 ** -4 + np.expm1(2 * e)) * (p @ np.abs(v)) + 2.0 ** -10 * np.abs(v).max() / 8
                want = f64(x[t]) + w_o @ o.ravel()
                bound = np.abs(w_o) @ tol.ravel() + 2.0 ** -6 * np.abs(want).max()
                err = np.abs(got[t] - want)
                assert (err <= bound).all(), (err / bound).max()
                # and as a whole the error is that of 8-bit keys and values: a few per cent
                assert np.linalg.norm(err) <= 2.0 ** -4 * np.linalg.norm(want)
                t += 1
