"""The attention weight of the 8-bit KV cache where query rows of one call differ (GPU): rows that give nothing, whatever
they hold, and rows of very different sizes.

Bound of a key's sum, with w_i = exp(s_i - lse_i) the weight of query row i on it: sum w_i e_i + 2^-21 sum w_i (the sum of
the rows, in any order) + 2^-22 of the result, where e_i = delta_i + 2^-22 (2 |s_i| + 2 |lse_i|) + 2^-19 and, bf16, delta_i =
2^-17 * scale * max|q_i| * sum|k| (queries as two E4M3 parts, exact to 2^-17.8 of the row's largest magnitude, and fp32
accumulation) or, fp32, 2^-20 * scale * sum |q_i k|.
"""
import numpy as np
import pytest
import torch

from block_diffusion_moe_dllm_b200 import binding as bd
from block_diffusion_moe_dllm_b200 import synth
from _util import to64
from test_gpu_kv8 import DEV, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bd.load()


def weigh(q, kc, ks, lse, P, S, lens=None):
    B, Lq, Hq, d = q.shape
    Hkv, cap = kc.shape[1], kc.shape[2]
    out = torch.full((B, Hkv, cap), -5.0, device=DEV)
    ws = bd.Workspace(1 << 16, DEV)
    bd.attn_mass_kv8(q, kc, ks, lse, None, out, B, Lq, Hq, Hkv, d, P, cap, S,
                     bd.BF16 if q.dtype == torch.bfloat16 else bd.F32, prefix_len=lens, ws=ws)
    assert bd.status_check(ws) == bd.OK
    return out


def log_sums(q, kv, P):
    """log sum exp(score) of every query over the first P keys, as the attention would give it, rounded to fp32."""
    B, Lq, Hq, d = q.shape
    G = Hq // kv.shape[1]
    s = np.einsum("bihd,bhjd->bihj", q, np.repeat(kv[:, :, :P], G, axis=1)) / np.sqrt(d)
    m = s.max(-1, keepdims=True)
    return s, (m[..., 0] + np.log(np.exp(s - m).sum(-1))).astype(np.float32)


# row tiles of 128 (bf16) and 64 (fp32): one with rows missing, several, and several in a cluster (fp32)
SHAPES = [("bf16", 2, 9, 8, 2, 128, 200, 16), ("bf16", 1, 300, 4, 2, 128, 140, 32), ("f32", 2, 9, 8, 2, 64, 100, 16),
          ("f32", 1, 80, 8, 1, 64, 70, 32)]


@pytest.mark.parametrize("dtype,B,Lq,Hq,Hkv,d,P,S", SHAPES)
@pytest.mark.parametrize("holds", [float("nan"), float("inf"), 1e30, 0.0])
def test_rows_without_keys_give_nothing_whatever_they_hold(dtype, B, Lq, Hq, Hkv, d, P, S, holds):
    """Rows whose log-sum-exp is -inf: the sums have the bits that the other rows give alone, beside rows of zeros."""
    t = synth.torch_dtype(dtype)
    kc, _, ks, _, kv, _ = make_cache(B, Hkv, P, d, S, 91)
    q = synth.normal((B, Lq, Hq, d), 1.5, 91, "q", DEV, t)
    s, lse = log_sums(to64(q), kv, P)
    none = synth.randint((B, Lq, Hq), 0, 3, 91, "none", DEV) == 0
    none[0, 0] = True
    lse = torch.where(none, -float("inf"), torch.from_numpy(lse).to(DEV))
    zero = torch.where(none[..., None], torch.zeros((), dtype=t, device=DEV), q)
    want = weigh(zero, kc, ks, lse, P, S)
    bad = zero.clone()
    bad[none] = holds
    bad[0, 0, 0] = 0
    bad[0, 0, 0, 3] = holds                                  # a single element of a row
    got = weigh(bad, kc, ks, lse, P, S)
    assert torch.isfinite(want).all() and torch.equal(got, want)
    l64 = to64(lse)
    w = np.where(l64[..., None] == -np.inf, 0, np.exp(s - np.where(l64 == -np.inf, 0, l64)[..., None]))
    total = w.sum(1).reshape(B, Hkv, -1, P).sum(2)
    assert np.allclose(to64(got)[:, :, :P], total, rtol=1e-3)


@pytest.mark.parametrize("dtype,B,Lq,Hq,Hkv,d,P,S", SHAPES)
@pytest.mark.parametrize("small", [2.0 ** -6, 2.0 ** -14])
def test_rows_of_different_sizes(dtype, B, Lq, Hq, Hkv, d, P, S, small):
    """One row in eight is 32 times as large as an ordinary one, the rest smaller: each row's weights are as exact as its
    own size allows."""
    t = synth.torch_dtype(dtype)
    G = Hq // Hkv
    kc, _, ks, _, kv, _ = make_cache(B, Hkv, P, d, S, 92)
    q = synth.normal((B, Lq, Hq, d), 1.0, 92, "q", DEV, torch.float32)
    large = (torch.arange(B * Lq * Hq, device=DEV) % 8 == 3).reshape(B, Lq, Hq, 1)
    q = torch.where(large, 32 * q, small * q).to(t)
    s, lse = log_sums(to64(q), kv, P)
    got = to64(weigh(q, kc, ks, torch.from_numpy(lse).to(DEV), P, S))[:, :, :P]
    l64, q64 = lse.astype(np.float64)[..., None], to64(q)
    w = np.exp(s - l64)
    kr = np.repeat(kv[:, :, :P], G, axis=1)
    if dtype == "bf16":
        delta = 2.0 ** -17 * np.abs(q64).max(-1)[..., None] * np.abs(kr).sum(-1)[:, None]
    else:
        delta = 2.0 ** -20 * np.einsum("bihd,bhjd->bihj", np.abs(q64), np.abs(kr))
    e = delta / np.sqrt(d) + 2.0 ** -22 * (2 * np.abs(s) + 2 * np.abs(l64)) + 2.0 ** -19
    group = lambda x: x.sum(1).reshape(B, Hkv, G, P).sum(2)
    want = group(w)
    bound = group(w * e) * 1.01 + 2.0 ** -21 * want + 2.0 ** -22 * want
    err = np.abs(got - want)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.3g} bounds"
