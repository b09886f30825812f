"""The 8-bit KV cache's attention against the fp64 formulas where values of very different sizes meet (GPU): own rows
that a query does not see, own rows of different sizes, and one key above all others.

Bounds, per element (u16 = 2^-8 and u32 = 2^-24: half a step of bf16 and fp32). With p_j the softmax weights, s_j the
scores, m the largest of them, a_j the largest magnitude of V row j and n the visible keys:
  score    bf16: 2^-17 * scale * (max|q| * sum|k_j| over the columns where q is not 0 + max|k_j| * sum|q| over those where
           k_j is not 0): queries and own keys are two E4M3 parts each, exact to 2^-17.8 of their row's largest magnitude,
           zeros exact, and fp32 accumulation adds less than 2^-18 of the first term. fp32: 2^-20 * scale * sum |q k_j|
           (128 products at most: 2^-24 of partial sums for each, of which 16 times their bound is allowed)
  weight   relative, e_j: the score's error, 2^-23 * (2 |s_j| + 2 |m| + 40) for the exponent (offsets of up to 40 in it are
           the V scales' logarithms), 2^-20 for the exponential and the sums
  output   u * |o| + sum p_j |v_j| (e_j + sum p e), and bf16's rounding of weights to f16: 2^-11 of sum p_j |v_j| (2^-7 of
           that more for weights rounded again when the reference moves), and n * 2^-25 * max_j(p_j a_j): a weight is
           4 w_j t_j / r with t_j the V scale of its key and r at most the largest w_j t_j; below 2^-14 its rounding error
           is 2^-25 at most, times V codes, which are at most twice a_j / t_j (own rows by the choice of their scale, the
           caches here by their codes' distribution), and twice that for weights rounded again
  lse      sum p e, and 2^-21 |lse| + 2^-20 for the logarithm and its sum with the reference
"""
import numpy as np
import pytest
import torch

from block_diffusion_moe_dllm_b200 import binding as bd
from block_diffusion_moe_dllm_b200 import synth
from oracle import kv8_oracle as K8
from _util import to64
from test_gpu_kv8 import DEV, codes64, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bd.load()


def attend(q, kc, vc, ks, vs, ko, vo, P, S, blk, lens=None, cap=None):
    """One call on whole tensors: output [B, Lq, Hq, d] and log-sum-exp."""
    B, Lq, Hq, d = q.shape
    Hkv = kc.shape[1]
    out = torch.full((B, Lq, Hq * d), float("nan"), dtype=q.dtype, device=DEV)
    lse = torch.full((B, Lq, Hq), float("nan"), device=DEV)
    dt = bd.BF16 if q.dtype == torch.bfloat16 else bd.F32
    ws = bd.Workspace(1 << 20, DEV)
    bd.block_attn_kv8(q, kc, vc, ks, vs, out, B, Lq, Hq, Hkv, d, P, cap or kc.shape[2], S, blk, dt, prefix_len=lens,
                      k_own=ko, v_own=vo, cap_own=0 if ko is None else ko.shape[2], lse=lse, ws=ws)
    assert bd.status_check(ws) == bd.OK
    return out.reshape(q.shape), lse


def check(out, lse, q, kv, vv, ko, vo, blk, rows=None):
    """out and lse of the query rows `rows` (all without it) within the bounds of this file. All in fp64 numpy but out, lse."""
    B, Lq, Hq, d = q.shape
    G = Hq // kv.shape[1]
    bf16 = out.dtype == torch.bfloat16
    got, gl = to64(out), to64(lse)
    u, scale = 2.0 ** -8 if bf16 else 2.0 ** -24, 1.0 / np.sqrt(d)
    for b in range(B):
        for i in range(Lq) if rows is None else rows:
            lim = 0 if ko is None else min(Lq, (i // blk + 1) * blk)
            for h in range(Hq):
                k, v = kv[b, h // G], vv[b, h // G]
                if lim:
                    k, v = np.concatenate([k, ko[b, h // G, :lim]]), np.concatenate([v, vo[b, h // G, :lim]])
                x = q[b, i, h]
                s = k @ x * scale
                m = s.max()
                w = np.exp(s - m)
                z = w.sum()
                p, l = w / z, m + np.log(z)
                o, oa = p @ v, p @ np.abs(v)
                ak, ax = np.abs(k), np.abs(x)
                if bf16:
                    e = 2.0 ** -17 * scale * (ax.max() * (ak @ (ax > 0)) + ak.max(1) * ((ak > 0) @ ax))
                    f16, lost = 2.0 ** -11 * (1 + 2.0 ** -7), len(s) * 2.0 ** -25 * (p * np.abs(v).max(1)).max()
                else:
                    e, f16, lost = 2.0 ** -20 * scale * (ak @ ax), 0.0, 0.0
                e = e + 2.0 ** -23 * (2 * np.abs(s) + 2 * abs(m) + 40) + 2.0 ** -20
                bound = u * np.abs(o) + (p * e) @ np.abs(v) + ((p @ e) + f16) * oa + lost + 1e-30
                err = np.abs(got[b, i, h] - o)
                assert np.all(err <= bound), f"row {b} {i} {h}: worst {np.max(err / bound):.3g} bounds"
                lb = p @ e + 2.0 ** -21 * abs(l) + 2.0 ** -20
                assert abs(gl[b, i, h] - l) <= lb, f"lse {b} {i} {h}: {abs(gl[b, i, h] - l) / lb:.3g} bounds"


def own_rows(shape, seed, tag, dtype):
    return synth.normal(shape, 1.0, seed, tag, DEV, dtype)


# ------------------------------------------------------------------------------------------------ own rows
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("P,Lq,blk,seen", [(0, 70, 1, 40), (140, 70, 1, 5), (33, 200, 1, 131), (16, 200, 4, 20)])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 30, 2.0 ** -40])
def test_own_rows_out_of_sight_change_nothing(dtype, d, P, Lq, blk, seen, size):
    """Causal queries before row `seen`: other rows from there on give the same bits, however large they are."""
    t = synth.torch_dtype(dtype)
    Hq = Hkv = 2
    kc, vc, ks, vs, kv, vv = make_cache(1, Hkv, max(P, 1), d, 16, 81)
    q, ko, vo = (own_rows(s, 81, x, t) for x, s in (("q", (1, Lq, Hq, d)), ("ko", (1, Hkv, Lq, d)), ("vo", (1, Hkv, Lq, d))))
    out, lse = attend(q, kc, vc, ks, vs, ko, vo, P, 16, blk)
    check(out, lse, to64(q), kv[:, :, :P], vv[:, :, :P], to64(ko), to64(vo), blk, range(0, seen, 7))
    k2, v2 = ko.clone(), vo.clone()
    k2[:, :, seen:] *= size
    v2[:, :, seen:] *= size
    out2, lse2 = attend(q, kc, vc, ks, vs, k2, v2, P, 16, blk)
    assert torch.equal(out[:, :seen], out2[:, :seen]) and torch.equal(lse[:, :seen], lse2[:, :seen])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("P,Lq,blk,seen", [(0, 70, 1, 40), (140, 70, 1, 5), (33, 200, 1, 131), (16, 200, 4, 20)])
@pytest.mark.parametrize("holds", [float("nan"), float("inf"), -float("inf")])
def test_own_rows_out_of_sight_may_hold_anything(dtype, d, P, Lq, blk, seen, holds):
    """A padded chunk: rows from `seen` on are infinite or NaN as a whole or in one element. The queries before give the bits
    that they give beside ordinary rows; those that see such a V row give NaN."""
    t = synth.torch_dtype(dtype)
    Hq = Hkv = 2
    kc, vc, ks, vs, _, _ = make_cache(1, Hkv, max(P, 1), d, 16, 86)
    q, ko, vo = (own_rows(s, 86, x, t) for x, s in (("q", (1, Lq, Hq, d)), ("ko", (1, Hkv, Lq, d)), ("vo", (1, Hkv, Lq, d))))
    out, lse = attend(q, kc, vc, ks, vs, ko, vo, P, 16, blk)
    k2, v2 = ko.clone(), vo.clone()
    v2[:, 0, seen:], k2[:, 0, seen:] = holds, holds
    v2[:, 1, seen, 9] = holds
    out2, lse2 = attend(q, kc, vc, ks, vs, k2, v2, P, 16, blk)
    assert torch.equal(out[:, :seen], out2[:, :seen]) and torch.equal(lse[:, :seen], lse2[:, :seen])
    assert torch.isnan(out2[:, seen:, 0]).all() and not torch.isfinite(out2[:, seen:, 1, 9]).any()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("P,Lq,blk", [(0, 32, 32), (100, 130, 1)])
def test_own_rows_of_different_sizes(dtype, d, P, Lq, blk):
    """Own values from 2^-12 to 2^4, ordinary own keys beside small ones and beside keys 2^14 times as large (in one column
    that the queries do not use): each row is held as exactly as it would be alone."""
    t = synth.torch_dtype(dtype)
    Hq, Hkv = 4, 2
    kc, vc, ks, vs, kv, vv = make_cache(1, Hkv, max(P, 1), d, 16, 82)
    q = own_rows((1, Lq, Hq, d), 82, "q", t)
    q[..., 5] = 0
    n = torch.arange(Lq, device=DEV)
    ev = n.mul(5).remainder(17).float() - 12
    ko = own_rows((1, Hkv, Lq, d), 82, "ko", torch.float32)
    ko[:, :, n % 4 == 1] *= 2.0 ** -10
    big = torch.zeros(d, device=DEV)
    big[5] = 2.0 ** 14
    ko[:, :, n % 4 == 2] = big
    ko = ko.to(t)
    vo = (own_rows((1, Hkv, Lq, d), 82, "vo", torch.float32) * torch.exp2(ev)[:, None]).to(t)
    out, lse = attend(q, kc, vc, ks, vs, ko, vo, P, 16, blk)
    check(out, lse, to64(q), kv[:, :, :P], vv[:, :, :P], to64(ko), to64(vo), blk)


# ------------------------------------------------------------------------------------------------ one key above all
@pytest.mark.parametrize("dtype,d,P", [("bf16", 128, 9000), ("f32", 64, 3000), ("bf16", 128, 33000)])
@pytest.mark.parametrize("gap", [4.0, 9.0, 13.0, 17.0])
def test_one_key_above_all_others(dtype, d, P, gap):
    """The first key's score lies `gap` above the rest of a long prefix, so that the others are together as heavy as it is,
    or each far below what f16 resolves beside it."""
    t = synth.torch_dtype(dtype)
    S, Hkv, Hq, Lq = 32, 1, 2, 2
    kc, vc, ks, vs, kv, vv = make_cache(1, Hkv, P, d, S, 83)
    q = own_rows((1, Lq, Hq, d), 83, "q", torch.float32) * 0.25
    # the first key is all +-64 * scale, with the queries' signs in a common half of the columns
    sign = torch.where(torch.arange(d, device=DEV) % 3 == 0, -1.0, 1.0)
    kc[0, 0, 0] = torch.where(sign > 0, 0x68, 0xE8).to(torch.uint8)         # +-64
    k0 = 64.0 * float(ks[0, 0, 0])
    q = (q + sign * gap * np.sqrt(d) / (d * k0)).to(t)
    kv = K8.values(codes64(kc), to64(ks), S)
    out, lse = attend(q, kc, vc, ks, vs, None, None, P, S, 1)
    check(out, lse, to64(q), kv, vv, None, None, 1)


def test_one_v_run_above_all_others():
    """A V run whose scale is 2^16 times the others' and whose codes fill one column: the other columns lose what the bound
    allows, n * 2^-25 of the largest weight times V, and no more; the log-sum-exp loses nothing."""
    B, Lq, Hq, Hkv, d, P, S = 1, 4, 4, 2, 128, 320, 32
    kc, vc, ks, vs, _, _ = make_cache(B, Hkv, P, d, S, 84)
    vc[:, :, 64:96] = 0
    vc[:, :, 64:96, 17] = 0x7E                                              # 448
    vs[:, :, 2] *= 2.0 ** 16
    kv, vv = K8.values(codes64(kc), to64(ks), S), K8.values(codes64(vc), to64(vs), S)
    q = own_rows((B, Lq, Hq, d), 84, "q", torch.bfloat16)
    out, lse = attend(q, kc, vc, ks, vs, None, None, P, S, 1)
    check(out, lse, to64(q), kv, vv, None, None, 1)


# ------------------------------------------------------------------------------------------------ no keys at all
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_queries_without_keys_are_zero_whatever_they_hold(dtype, d, bad):
    t = synth.torch_dtype(dtype)
    B, Lq, Hq, Hkv, P, S = 3, 5, 4, 2, 200, 32
    kc, vc, ks, vs, kv, vv = make_cache(B, Hkv, P, d, S, 85)
    q = own_rows((B, Lq, Hq, d), 85, "q", t)
    q[1, 2:, 1, 7] = bad
    q[1, 3] = bad
    lens = torch.tensor([P, 0, 131], dtype=torch.int32, device=DEV)
    out, lse = attend(q, kc, vc, ks, vs, None, None, P, S, 1, lens=lens)
    assert not out[1].any() and torch.all(lse[1] == -float("inf"))
    for b, n in ((0, P), (2, 131)):
        check(out[b: b + 1], lse[b: b + 1], to64(q[b: b + 1]), kv[b: b + 1, :, :n], vv[b: b + 1, :, :n], None, None, 1)
