"""Parity of the 8-bit KV cache operators with the fp64 oracle (GPU): store, block attention, attention weight,
eviction, and a run of them together.

Tolerances, per element, from the arithmetic of the kernels (u16 = 2^-8 and u32 = 2^-24: half a step of bf16 and fp32):
  score    delta = 2^-17 * scale * max|q| * sum|k|: the queries are held as two E4M3 parts of a common power-of-two
           scale per row that brings max|q| into [224, 448], so a part's rounding error is at most half the smallest
           E4M3 step, 2^-10, that is 2^-17.8 of max|q|; fp32 accumulation adds less than 2^-18 of the same sum
  weight   exp(score - max): relative error at most delta (twice: score and maximum) + |exponent| * 2^-22 + 2^-20
  output   rounding of the result (u16 or u32), the weights' error and their f16 rounding (2^-11) against sum p |v|
  lse      delta + rounding of a logarithm and of the maximum in fp32
"""
import numpy as np
import pytest
import torch

from block_diffusion_moe_dllm_b200 import binding as bd
from block_diffusion_moe_dllm_b200 import synth
from oracle import kv8_oracle as K8
from _util import to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": bd.BF16, "f32": bd.F32}
NAN_CODE = 0x7F


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bd.load()


def cdiv(a, b):
    return -(-a // b)


def codes64(t):
    """Values of a uint8 code tensor."""
    return K8.e4m3_values()[t.cpu().numpy()]


def same(got, want):
    return np.array_equal(got, want, equal_nan=True)


def rows_like_tokens(shape, seed, tag, dtype):
    x = synth.normal(shape, 1.0, seed, tag, DEV, torch.float32)
    return (x * torch.exp(0.5 * synth.normal((*shape[:-1], 1), 1.0, seed, tag + "m", DEV, torch.float32))).to(dtype)


def make_cache(B, Hkv, cap, d, S, seed, pow2=True):
    """A cache of random codes (no NaN codes) and scales; values about N(0, 1). Returns code tensors, scale tensors and
    the values in fp64."""
    out = []
    for tag in ("k", "v"):
        c = (synth.normal((B, Hkv, cap, d), 24.0, seed, tag + "c", DEV, torch.float32)).to(torch.float8_e4m3fn)
        e = synth.randint((B, Hkv, cdiv(cap, S)), -6, -3, seed, tag + "e", DEV).float()
        sc = torch.exp2(e) if pow2 else torch.exp2(e) * synth.uniform(e.shape, 0.6, 1.5, seed, tag + "s", DEV)
        out += [c.view(torch.uint8).contiguous(), sc.contiguous()]
    kc, ks, vc, vs = out
    val = [K8.values(codes64(c), to64(s), S) for c, s in ((kc, ks), (vc, vs))]
    return kc, vc, ks, vs, val[0], val[1]


# ------------------------------------------------------------------------------------------------ store
@pytest.mark.parametrize("dtype,B,Hkv,d,n,S", [
    ("bf16", 1, 1, 128, 1, 32), ("bf16", 2, 4, 128, 32, 32), ("bf16", 3, 2, 128, 77, 16), ("bf16", 1, 3, 64, 130, 64),
    ("bf16", 2, 1, 16, 300, 128), ("bf16", 1, 2, 112, 33, 128), ("f32", 2, 2, 64, 50, 16), ("f32", 1, 1, 128, 129, 128),
    ("f32", 1, 5, 80, 31, 64), ("bf16", 5, 4, 128, 1000, 64)])
def test_store(dtype, B, Hkv, d, n, S):
    t = synth.torch_dtype(dtype)
    cap_src, src_row = n + 5, 3
    cap = cdiv(n, S) * S + 2 * S + 7
    k = rows_like_tokens((B, Hkv, cap_src, d), 1, "k", t)
    v = rows_like_tokens((B, Hkv, cap_src, d), 1, "v", t)
    rows = torch.tensor([(b % 3) * S for b in range(B)], dtype=torch.int32, device=DEV)
    codes = [torch.full((B, Hkv, cap, d), 0xA5, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scale = [torch.full((B, Hkv, cdiv(cap, S)), -7.0, device=DEV) for _ in range(2)]
    bd.kv8_store(k, v, *codes, *scale, B, Hkv, d, n, cap_src, cap, S, DT[dtype], src_row=src_row, dst_rows=rows)
    for x, c, s in ((k, codes[0], scale[0]), (v, codes[1], scale[1])):
        wc, ws = K8.store(to64(x)[:, :, src_row: src_row + n], S)
        want_c = np.full((B, Hkv, cap, d), K8.e4m3_values()[0xA5])
        want_s = np.full((B, Hkv, cdiv(cap, S)), -7.0)
        for b in range(B):
            r0 = (b % 3) * S
            want_c[b, :, r0: r0 + n] = wc[b]
            want_s[b, :, r0 // S: r0 // S + ws.shape[-1]] = ws[b]
        assert same(to64(s), want_s)
        assert same(codes64(c), want_c)       # bit for bit, rows outside the call untouched


def test_store_special_values():
    """Zeros, infinities, NaN, the largest and the smallest magnitudes; -0 keeps its sign in the code."""
    B, Hkv, d, n, S = 1, 1, 128, 6 * 16, 16
    x = synth.normal((B, Hkv, n, d), 1.0, 2, "sp", DEV, torch.float32)
    x[0, 0, 0:16] = 0
    x[0, 0, 16, 5], x[0, 0, 17, 6], x[0, 0, 18, 7] = float("inf"), float("-inf"), float("nan")
    x[0, 0, 32:48] *= 1e-30
    x[0, 0, 48, 0] = 3.3e38
    x[0, 0, 64:80] = 448.0 * 2.0 ** -5
    x[0, 0, 80:96] = -0.0
    x[0, 0, 80, 0] = 1.75
    for dtype, t in (("f32", torch.float32), ("bf16", torch.bfloat16)):
        k = x.to(t)
        kc, vc = (torch.zeros((B, Hkv, n, d), dtype=torch.uint8, device=DEV) for _ in range(2))
        ks, vs = (torch.zeros((B, Hkv, n // S), device=DEV) for _ in range(2))
        bd.kv8_store(k, k, kc, vc, ks, vs, B, Hkv, d, n, n, n, S, DT[dtype])
        wc, ws = K8.store(to64(k), S)
        assert same(to64(ks), ws) and same(codes64(kc), wc) and torch.equal(kc, vc) and torch.equal(ks, vs)
        assert kc[0, 0, 81, 3].item() == 0x80


def test_store_gathers_positions_and_leaves_bad_rows():
    """src_pos as a retention list (out-of-range entries store zeros); a batch row whose dst_rows entry does not start a
    run, is negative or leaves no room is left as it was."""
    B, Hkv, d, n, S, cap_src, cap = 5, 2, 128, 40, 32, 64, 128
    k = rows_like_tokens((B, Hkv, cap_src, d), 4, "k", torch.bfloat16)
    v = rows_like_tokens((B, Hkv, cap_src, d), 4, "v", torch.bfloat16)
    pos = synth.randint((B, n + 3), 0, cap_src, 4, "pos", DEV)
    pos[0, 1], pos[0, 2] = -1, cap_src
    rows = torch.tensor([32, 8, -32, 96, 64], dtype=torch.int32, device=DEV)
    codes = [torch.full((B, Hkv, cap, d), 0x11, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scale = [torch.full((B, Hkv, cap // S), 3.0, device=DEV) for _ in range(2)]
    bd.kv8_store(k, v, *codes, *scale, B, Hkv, d, n, cap_src, cap, S, bd.BF16, src_pos=pos, dst_rows=rows,
                 pos_stride=n + 3)
    p = pos.cpu().numpy()[:, :n]
    ok = (p >= 0) & (p < cap_src)
    for x, c, s in ((k, codes[0], scale[0]), (v, codes[1], scale[1])):
        want_c, want_s = np.full((B, Hkv, cap, d), K8.e4m3_values()[0x11]), np.full((B, Hkv, cap // S), 3.0)
        for b, r0 in ((0, 32), (4, 64)):
            src = to64(x)[b][:, np.where(ok[b], p[b], 0)] * ok[b][None, :, None]
            wc, ws = K8.store(src, S)
            want_c[b, :, r0: r0 + n], want_s[b, :, r0 // S: r0 // S + 2] = wc, ws
        assert same(codes64(c), want_c) and same(to64(s), want_s)


# ------------------------------------------------------------------------------------------------ attention
def attn_inputs(dtype, B, Lq, Hq, Hkv, d, P, S, lens, own, seed, cap=None, pow2=True, q_std=1.5):
    t = synth.torch_dtype(dtype)
    cap = cap or P
    kc, vc, ks, vs, kv, vv = make_cache(B, Hkv, max(cap, 1), d, S, seed, pow2)
    q = synth.normal((B, Lq, Hq, d), q_std, seed, "q", DEV, t)
    ko = rows_like_tokens((B, Hkv, Lq + 3, d), seed, "ko", t) if own else None
    vo = rows_like_tokens((B, Hkv, Lq + 3, d), seed, "vo", t) if own else None
    if own:
        ko[:, :, Lq:], vo[:, :, Lq:] = float("nan"), float("nan")      # rows the call must not read
    if lens is not None:
        # what lies past a row's length: NaN codes, and NaN scales for runs that lie past it as a whole
        for b in range(B):
            n = max(0, min(int(lens[b]), P))
            for c, s in ((kc, ks), (vc, vs)):
                c[b, :, n:] = NAN_CODE
                s[b, :, cdiv(n, S):] = float("nan")
    return q, kc, vc, ks, vs, kv, vv, ko, vo


def check_attn(dtype, out, lse, q, kv, vv, lens, ko, vo, Lq, blk, d):
    o, l, oa, big = K8.attention(to64(q), kv, vv, lens, None if ko is None else to64(ko)[:, :, :Lq],
                                 None if vo is None else to64(vo)[:, :, :Lq], blk)
    delta = 2.0 ** -17 * big
    eps = 2 * delta + 2 * big * 2.0 ** -22 + 2.0 ** -20
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    f16 = 2.0 ** -11 if dtype == "bf16" else 0.0
    got = to64(out).reshape(o.shape)
    bound = u * np.abs(o) + (2 * eps[..., None] + f16 + 2.0 ** -20) * oa + 1e-30
    err = np.abs(got - o)
    assert np.all(np.isfinite(got))
    assert np.all(err <= bound), f"{int((err > bound).sum())} outputs, worst {np.max(err / bound):.3g} bounds"
    empty = l == -np.inf
    gl = to64(lse)
    assert np.array_equal(gl == -np.inf, empty)
    le = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, l))
    lb = delta + 2.0 ** -20 + 2.0 ** -21 * np.abs(np.where(empty, 0, l))
    assert np.all(le <= lb), f"lse: worst {np.max(le / lb):.3g} bounds"
    return l


ATTN = [
    # dtype, B, Lq, Hq, Hkv, d, P, S, blk, lens, own
    ("f32", 1, 16, 4, 4, 64, 64, 16, 16, None, True), ("f32", 3, 16, 4, 4, 64, 300, 16, 16, (300, 0, 129), True),
    ("f32", 2, 5, 6, 2, 80, 100, 32, 2, (1, 99), True), ("f32", 1, 1, 7, 1, 128, 2000, 128, 1, (1999,), True),
    ("f32", 2, 33, 3, 1, 16, 40, 64, 8, (0, 40), False), ("f32", 1, 70, 2, 2, 32, 0, 16, 32, None, True),
    ("bf16", 1, 32, 16, 4, 128, 1024, 32, 32, None, True), ("bf16", 1, 1, 4, 4, 128, 1, 16, 1, None, False),
    ("bf16", 2, 32, 16, 4, 128, 300, 32, 32, (300, 171), True), ("bf16", 3, 32, 8, 8, 128, 260, 16, 32, (0, 1, 257), True),
    ("bf16", 4, 1, 28, 4, 128, 515, 16, 1, (515, 0, 128, 127), True), ("bf16", 2, 7, 10, 2, 128, 130, 64, 4, (129, 130), True),
    ("bf16", 1, 200, 4, 1, 128, 384, 128, 32, (383,), True), ("bf16", 1, 131, 3, 3, 128, 0, 16, 1, None, True),
    ("bf16", 2, 16, 48, 2, 128, 140, 32, 16, (140, 13), False), ("bf16", 1, 300, 16, 2, 128, 70, 16, 4096, None, True),
    ("bf16", 9, 4, 4, 2, 128, 1100, 64, 4, (1100, 3, 0, 640, 1024, 1, 128, 129, 900), True),
    ("bf16", 8, 260, 16, 4, 128, 200, 32, 32, (200, 0, 129, 128, 1, 77, 200, 3), True),    # many units a CTA, several
    ("bf16", 300, 1, 4, 4, 128, 0, 16, 1, None, True),                                    # own tiles in a row
    ("bf16", 200, 1, 8, 4, 128, 130, 16, 1, tuple(i % 3 * 65 for i in range(200)), False),
    ("bf16", 1, 2, 16, 1, 128, 9000, 128, 1, (8999,), True), ("bf16", 40, 1, 1, 1, 128, 50, 16, 1, tuple(range(40)), True)]


@pytest.mark.parametrize("dtype,B,Lq,Hq,Hkv,d,P,S,blk,lens,own", ATTN)
def test_block_attn_kv8(dtype, B, Lq, Hq, Hkv, d, P, S, blk, lens, own):
    cap = P + 37
    q, kc, vc, ks, vs, kv, vv, ko, vo = attn_inputs(dtype, B, Lq, Hq, Hkv, d, P, S, lens if lens else (P,) * B, own, 7, cap)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV) if lens else None
    out = torch.full((B, Lq, Hq * d), float("nan"), dtype=q.dtype, device=DEV)
    lse = torch.full((B, Lq, Hq), float("nan"), device=DEV)
    need_ws = bd.Workspace(1 << 20, DEV)
    bd.block_attn_kv8(q, kc, vc, ks, vs, out, B, Lq, Hq, Hkv, d, P, cap, S, blk, DT[dtype], prefix_len=ld, k_own=ko,
                      v_own=vo, cap_own=Lq + 3, lse=lse, ws=need_ws)
    assert bd.status_check(need_ws) == bd.OK
    check_attn(dtype, out, lse, q, kv, vv, lens if lens else (P,) * B, ko, vo, Lq, blk, d)
    # without the log-sum-exp, and again: the same bits
    out2 = torch.full_like(out, float("nan"))
    bd.block_attn_kv8(q, kc, vc, ks, vs, out2, B, Lq, Hq, Hkv, d, P, cap, S, blk, DT[dtype], prefix_len=ld, k_own=ko,
                      v_own=vo, cap_own=Lq + 3, ws=need_ws)
    assert torch.equal(out, out2)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_block_attn_kv8_scales_of_any_quantiser(dtype, d):
    """Scales that are no powers of two, a scale argument, lengths outside [0, P] read clamped, peaked scores."""
    B, Lq, Hq, Hkv, P, S = 3, 8, 8, 2, 200, 16
    lens = (200, 0, 150)
    q, kc, vc, ks, vs, kv, vv, ko, vo = attn_inputs(dtype, B, Lq, Hq, Hkv, d, P, S, lens, True, 11, pow2=False, q_std=6.0)
    ld = torch.tensor((999, -5, 150), dtype=torch.int32, device=DEV)
    out = torch.empty((B, Lq, Hq * d), dtype=q.dtype, device=DEV)
    lse = torch.empty((B, Lq, Hq), device=DEV)
    bd.block_attn_kv8(q, kc, vc, ks, vs, out, B, Lq, Hq, Hkv, d, P, P, S, 8, DT[dtype], prefix_len=ld, k_own=ko, v_own=vo,
                      cap_own=Lq + 3, lse=lse, scale=1.0 / np.sqrt(d))
    check_attn(dtype, out, lse, q, kv, vv, lens, ko, vo, Lq, 8, d)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_block_attn_kv8_wide_ranges(dtype, d):
    """V runs whose scales differ by 2^40, an all-zero run with the smallest scale, tiny and huge queries."""
    B, Lq, Hq, Hkv, P, S = 1, 4, 4, 2, 256, 32
    q, kc, vc, ks, vs, kv, vv, ko, vo = attn_inputs(dtype, B, Lq, Hq, Hkv, d, P, S, (P,), True, 12)
    vs[:, :, 3] *= 2.0 ** 20
    vs[:, :, 5] *= 2.0 ** -20
    vc[:, :, 0:32], vs[:, :, 0] = 0, 2.0 ** -64
    kc[:, :, 32:64], ks[:, :, 1] = 0, 2.0 ** -64
    q[0, 1] *= 2.0 ** -40
    q[0, 2, 0] = 0
    kv, vv = K8.values(codes64(kc), to64(ks), S), K8.values(codes64(vc), to64(vs), S)
    out = torch.empty((B, Lq, Hq * d), dtype=q.dtype, device=DEV)
    lse = torch.empty((B, Lq, Hq), device=DEV)
    bd.block_attn_kv8(q, kc, vc, ks, vs, out, B, Lq, Hq, Hkv, d, P, P, S, 4, DT[dtype], k_own=ko, v_own=vo, cap_own=Lq + 3,
                      lse=lse)
    check_attn(dtype, out, lse, q, kv, vv, (P,), ko, vo, Lq, 4, d)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_block_attn_kv8_nan_queries_stay_their_own(dtype, d):
    """A NaN or infinite query, and a NaN in a visible key, make NaN where they are seen and nothing elsewhere."""
    B, Lq, Hq, Hkv, P, S = 2, 4, 4, 2, 130, 32
    q, kc, vc, ks, vs, kv, vv, ko, vo = attn_inputs(dtype, B, Lq, Hq, Hkv, d, P, S, (P, P), True, 13)
    q[0, 1, 0, 5], q[0, 2, 3, 7] = float("nan"), float("inf")
    kc[1, 1, 17, 3] = NAN_CODE
    out = torch.empty((B, Lq, Hq * d), dtype=q.dtype, device=DEV)
    bd.block_attn_kv8(q, kc, vc, ks, vs, out, B, Lq, Hq, Hkv, d, P, P, S, 4, DT[dtype], k_own=ko, v_own=vo, cap_own=Lq + 3)
    bad = torch.isnan(out.reshape(B, Lq, Hq, d))
    want = torch.zeros((B, Lq, Hq), dtype=torch.bool, device=DEV)
    want[0, 1, 0] = want[0, 2, 3] = True
    want[1, :, 2:] = True
    assert torch.equal(bad.any(-1), want) and torch.equal(bad.all(-1), want)


# ------------------------------------------------------------------------------------------------ attention weight
MASS = [("f32", 2, 5, 6, 2, 80, 100, 32, (1, 99)), ("f32", 1, 33, 3, 1, 16, 70, 16, None),
        ("bf16", 1, 32, 16, 4, 128, 300, 32, None), ("bf16", 3, 1, 28, 4, 128, 515, 16, (515, 0, 129)),
        ("bf16", 2, 40, 16, 2, 128, 260, 64, (257, 128)), ("bf16", 1, 300, 5, 1, 128, 150, 128, (149,)),
        ("bf16", 20, 3, 4, 4, 128, 140, 16, tuple(range(121, 141))),
        ("bf16", 40, 70, 8, 2, 128, 700, 64, tuple(i * 17 % 701 for i in range(40))),   # several row and key tiles a CTA
        ("bf16", 1, 1, 2, 2, 128, 1, 16, None)]


@pytest.mark.parametrize("dtype,B,Lq,Hq,Hkv,d,P,S,lens", MASS)
@pytest.mark.parametrize("start", ["zeros", "same", "other"])
def test_attn_mass_kv8(dtype, B, Lq, Hq, Hkv, d, P, S, lens, start):
    cap = P + 21
    ln = lens if lens else (P,) * B
    q, kc, vc, ks, vs, kv, vv, _, _ = attn_inputs(dtype, B, Lq, Hq, Hkv, d, P, S, ln, False, 21, cap)
    _, l, _, big = K8.attention(to64(q), kv, vv, ln, None, None, 1)
    l = np.where(l == -np.inf, l, l + 0.25)
    lse = torch.from_numpy(l.astype(np.float32)).to(DEV)
    lse[0, 0, 0] = float("-inf")                                     # a row without keys adds nothing
    l = to64(lse)
    mass = synth.uniform((B, Hkv, cap), 0.0, 3.0, 21, "mass", DEV)
    old, decay = to64(mass), 0.75
    mass_out = mass if start == "same" else torch.full_like(mass, -5.0)
    bd.attn_mass_kv8(q, kc, ks, lse, None if start == "zeros" else mass, mass_out, B, Lq, Hq, Hkv, d, P, cap, S, DT[dtype],
                     prefix_len=torch.tensor(lens, dtype=torch.int32, device=DEV) if lens else None, decay=decay)
    base = old if start == "same" else np.full(old.shape, -5.0)
    want = K8.mass(to64(q), kv, ln, l, None if start == "zeros" else old, base, decay)
    add = want - np.where(np.arange(cap) < np.array(ln)[:, None, None], 0 if start == "zeros" else decay * old, base)
    fin = np.where(l == -np.inf, 0, l)
    eps = (2.0 ** -17 * big + (2 * big + np.abs(fin)) * 2.0 ** -22 + 2.0 ** -19).max()
    bound = 1.01 * eps * np.abs(add) + 2.0 ** -22 * np.abs(want) + 1e-30
    got = to64(mass_out)
    past = np.broadcast_to(np.arange(cap) >= np.array(ln)[:, None, None], got.shape)
    assert np.array_equal(got[past], base[past])
    err = np.abs(got - want)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.3g} bounds"


# few keys and several row tiles of 64: 8, 5, 3 and 2 of them shared by clusters of 8, 4, 2 and 2 CTAs (sums of at most 4
# rows a tile, 16 threads and 8 CTAs: below 2^-19 of rounding, as in the bound above)
@pytest.mark.parametrize("B,Lq,Hq,Hkv,d,P,S,lens", [(1, 32, 16, 1, 64, 70, 16, None), (3, 20, 32, 2, 128, 99, 32, (99, 0, 33)),
                                                    (1, 65, 2, 1, 80, 40, 64, None), (2, 32, 20, 5, 32, 31, 16, (31, 1))])
def test_attn_mass_kv8_f32_row_tiles(B, Lq, Hq, Hkv, d, P, S, lens):
    test_attn_mass_kv8("f32", B, Lq, Hq, Hkv, d, P, S, lens, "same")


# ------------------------------------------------------------------------------------------------ eviction
EVICT = [(1, 1, 128, 1, 16, 1, 0, 0, None), (2, 4, 128, 300, 32, 150, 4, 64, (300, 171)),
         (3, 2, 64, 257, 16, 100, 0, 0, (257, 0, 99)), (2, 3, 128, 1500, 64, 1400, 1, 1, (1500, 1401)),
         (1, 2, 32, 5000, 128, 333, 8, 100, (4999,)), (2, 2, 128, 90, 32, 200, 2, 2, (90, 1)),
         (1, 1, 16, 2100, 16, 64, 64, 0, None), (1, 2, 16, 20001, 64, 7000, 3, 5, (19999,)),
         (1, 1, 16, 270000, 128, 30000, 0, 0, None),     # keys in the workspace
         (2, 1, 128, 40, 128, 39, 0, 39, (40, 38))]


@pytest.mark.parametrize("B,Hkv,d,P,S,keep,first,last,lens", EVICT)
@pytest.mark.parametrize("per_head", [0, 1])
@pytest.mark.parametrize("ties", [False, True])
def test_kv8_evict(B, Hkv, d, P, S, keep, first, last, lens, per_head, ties):
    cap, cap_out = P + 11, keep + 5
    kc, vc, ks, vs, _, _ = make_cache(B, Hkv, cap, d, S, 31, pow2=not ties)
    if ties:
        mass = synth.randint((B, Hkv, cap), 0, 3, 31, "m", DEV).float()
    else:
        mass = torch.exp(2 * synth.normal((B, Hkv, cap), 1.0, 31, "m", DEV, torch.float32))
    mass[:, :, 0::7] = 0
    mass[0, 0, min(3, P - 1)] = float("nan")
    mass[0, 0, min(4, P - 1)] = -2.0
    Hs = Hkv if per_head else 1
    pos = synth.randint((B, Hs, cap), 0, 1 << 30, 31, "p", DEV) if ties else None
    ln = lens if lens else (P,) * B
    o = [torch.full((B, Hkv, cap_out, d), 0x33, dtype=torch.uint8, device=DEV) for _ in range(2)]
    s = [torch.full((B, Hkv, cdiv(cap_out, S)), -1.0, device=DEV) for _ in range(2)]
    mo = torch.full((B, Hkv, cap_out), -2.0, device=DEV)
    kp = torch.full((B, Hs, cap_out), -3, dtype=torch.int32, device=DEV)
    lo = torch.full((B,), -4, dtype=torch.int32, device=DEV)
    bd.kv8_evict(kc, vc, ks, vs, mass, *o, *s, mo, kp, lo, B, Hkv, d, P, cap, keep, cap_out, S, first, last, per_head,
                 prefix_len=torch.tensor(lens, dtype=torch.int32, device=DEV) if lens else None, pos=pos)
    m64 = to64(mass)
    assert lo.tolist() == [min(n, keep) for n in ln]
    for b in range(B):
        for h in range(Hkv):
            hs = h if per_head else 0
            rows = K8.select(m64[b, h: h + 1] if per_head else m64[b], ln[b], keep, first, last)
            c = len(rows)
            want = rows if pos is None else pos[b, hs].cpu().numpy()[rows]
            assert np.array_equal(kp[b, hs].cpu().numpy()[:c], want) and torch.all(kp[b, hs, c:] == -3)
            assert same(to64(mo)[b, h, :c], m64[b, h, rows]) and torch.all(mo[b, h, c:] == -2)
            for src, sc, dst, sd in ((kc, ks, o[0], s[0]), (vc, vs, o[1], s[1])):
                if ties:     # ratios that are no powers of two: the fp32 product may round to the other neighbour
                    r64 = to64(sc)[b, h][rows // S]
                    new = np.array([r64[i * S: (i + 1) * S].max() for i in range(cdiv(c, S))])
                    v = codes64(src)[b, h][rows] * r64[:, None]
                    g = codes64(dst)[b, h, :c] * np.repeat(new, S)[:c, None]
                    step = np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10 * np.repeat(new, S)[:c, None])
                    assert np.all(np.abs(g - v) <= step * (1 + 2.0 ** -20))
                    wn = new
                else:
                    wc, wn = K8.evict_rows(codes64(src)[b, h], to64(sc)[b, h], rows, S)
                    assert same(codes64(dst)[b, h, :c], wc)
                assert same(to64(sd)[b, h, : len(wn)], wn)
                assert torch.all(dst[b, h, c:] == 0x33) and torch.all(sd[b, h, len(wn):] == -1)


def test_empty_calls():
    """No rows to store, no prefix to attend to, to weigh or to evict: nothing is written but zeros for the queries."""
    B, Hkv, d, S = 2, 2, 128, 16
    c = [torch.full((B, Hkv, 16, d), 7, dtype=torch.uint8, device=DEV) for _ in range(4)]
    s = [torch.full((B, Hkv, 1), 7.0, device=DEV) for _ in range(4)]
    x = torch.zeros((B, Hkv, 16, d), dtype=torch.bfloat16, device=DEV)
    bd.kv8_store(x, x, c[0], c[1], s[0], s[1], B, Hkv, d, 0, 16, 16, S, bd.BF16)
    q = synth.normal((B, 3, 4, d), 1.0, 91, "q", DEV)
    out, lse = torch.full((B, 3, 4 * d), 5.0, dtype=torch.bfloat16, device=DEV), torch.zeros((B, 3, 4), device=DEV)
    bd.block_attn_kv8(q, c[0], c[1], s[0], s[1], out, B, 3, 4, Hkv, d, 0, 16, S, 1, bd.BF16, lse=lse)
    assert not out.any() and torch.all(lse == -float("inf"))
    mass, m2 = torch.full((B, Hkv, 16), 3.0, device=DEV), torch.full((B, Hkv, 16), 3.0, device=DEV)
    bd.attn_mass_kv8(q, c[0], s[0], lse, None, mass, B, 3, 4, Hkv, d, 0, 16, S, bd.BF16)
    pos, lens = torch.full((B, 1, 16), 9, dtype=torch.int32, device=DEV), torch.full((B,), 9, dtype=torch.int32, device=DEV)
    bd.kv8_evict(c[0], c[1], s[0], s[1], mass, c[2], c[3], s[2], s[3], m2, pos, lens, B, Hkv, d, 0, 16, 4, 16, S)
    assert lens.tolist() == [0, 0] and torch.all(pos == 9)
    assert all(torch.all(y == 7) for y in c + s) and torch.all(mass == 3) and torch.all(m2 == 3)


# ------------------------------------------------------------------------------------------------ together
def test_serving_run():
    """A prompt stored, a block attending over it, its weights accumulated, the prefix evicted to half, the block's own
    rows stored behind what was kept, and the next block attending over that: every stage against the oracle's own chain
    (its positions, its codes), on a side stream and with one workspace, and again as a captured graph."""
    B, L, Hq, Hkv, d, S, P = 2, 32, 16, 4, 128, 32, 320
    lens = (320, 224)
    bf = torch.bfloat16
    kp, vp = (rows_like_tokens((B, Hkv, P, d), 41, x, bf) for x in ("kp", "vp"))
    q1, q2 = (synth.normal((B, L, Hq, d), 1.5, 41, x, DEV) for x in ("q1", "q2"))
    k1, v1, k2, v2 = (rows_like_tokens((B, Hkv, L, d), 41, x, bf) for x in ("k1", "v1", "k2", "v2"))

    # the oracle's chain
    ck, sk = K8.store(to64(kp), S)
    cv, sv = K8.store(to64(vp), S)
    o1, l1, _, _ = K8.attention(to64(q1), K8.values(ck, sk, S), K8.values(cv, sv, S), lens, to64(k1), to64(v1), L)
    m1 = K8.mass(to64(q1), K8.values(ck, sk, S), lens, l1, None, np.zeros((B, Hkv, P)))
    # a count whose border has a clear gap for every batch row (weights differ there by 0.1 % at least)
    for keep in range(150, 220):
        gaps = []
        for b in range(B):
            t = m1[b, :, 4: lens[b] - 32].sum(0)
            t = np.sort(t)[::-1]
            gaps.append(t[keep - 37] / t[keep - 36] - 1)
        if keep % 32 == 0 and min(gaps) > 1e-3:
            break
    assert keep % 32 == 0 and min(gaps) > 1e-3
    cap2 = keep + L
    rows = [K8.select(m1[b], lens[b], keep, 4, 32) for b in range(B)]
    ck2, cv2 = np.zeros((B, Hkv, cap2, d)), np.zeros((B, Hkv, cap2, d))
    sk2, sv2 = np.ones((B, Hkv, cdiv(cap2, S))), np.ones((B, Hkv, cdiv(cap2, S)))
    for b in range(B):
        for h in range(Hkv):
            for c, s, c2, s2, own in ((ck, sk, ck2, sk2, k1), (cv, sv, cv2, sv2, v1)):
                c2[b, h, :keep], s2[b, h, : keep // S] = K8.evict_rows(c[b, h], s[b, h], rows[b], S)
                c2[b, h, keep:], s2[b, h, keep // S:] = K8.store(to64(own)[b, h], S)

    dev = dict(dtype=torch.uint8, device=DEV)
    kc, vc = torch.zeros((B, Hkv, P, d), **dev), torch.zeros((B, Hkv, P, d), **dev)
    ks, vs = torch.zeros((B, Hkv, P // S), device=DEV), torch.zeros((B, Hkv, P // S), device=DEV)
    kc2, vc2 = torch.zeros((B, Hkv, cap2, d), **dev), torch.zeros((B, Hkv, cap2, d), **dev)
    ks2, vs2 = torch.ones((B, Hkv, cdiv(cap2, S)), device=DEV), torch.ones((B, Hkv, cdiv(cap2, S)), device=DEV)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out1, out2 = torch.zeros((B, L, Hq * d), dtype=bf, device=DEV), torch.zeros((B, L, Hq * d), dtype=bf, device=DEV)
    lse1, lse2 = torch.zeros((B, L, Hq), device=DEV), torch.zeros((B, L, Hq), device=DEV)
    mass, mass2 = torch.zeros((B, Hkv, P), device=DEV), torch.zeros((B, Hkv, cap2), device=DEV)
    pos, len2 = torch.zeros((B, 1, cap2), dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    ws = bd.Workspace(32 << 20, DEV)

    def chain():
        bd.kv8_store(kp, vp, kc, vc, ks, vs, B, Hkv, d, P, P, P, S, bd.BF16)
        bd.block_attn_kv8(q1, kc, vc, ks, vs, out1, B, L, Hq, Hkv, d, P, P, S, L, bd.BF16, prefix_len=ld, k_own=k1, v_own=v1,
                          cap_own=L, lse=lse1, ws=ws)
        bd.attn_mass_kv8(q1, kc, ks, lse1, None, mass, B, L, Hq, Hkv, d, P, P, S, bd.BF16, prefix_len=ld, ws=ws)
        bd.kv8_evict(kc, vc, ks, vs, mass, kc2, vc2, ks2, vs2, mass2, pos, len2, B, Hkv, d, P, P, keep, cap2, S, 4, 32,
                     prefix_len=ld, ws=ws)
        bd.kv8_store(k1, v1, kc2, vc2, ks2, vs2, B, Hkv, d, L, L, cap2, S, bd.BF16, dst_rows=len2)
        bd.block_attn_kv8(q2, kc2, vc2, ks2, vs2, out2, B, L, Hq, Hkv, d, cap2, cap2, S, L, bd.BF16, k_own=k2, v_own=v2,
                          cap_own=L, lse=lse2, ws=ws)

    def check():
        assert same(codes64(kc), ck) and same(to64(vs), sv)
        check_attn("bf16", out1, lse1, q1, K8.values(ck, sk, S), K8.values(cv, sv, S), lens, k1, v1, L, L, d)
        for b in range(B):
            assert np.array_equal(pos[b, 0, :keep].cpu().numpy(), rows[b])
        assert len2.tolist() == [keep] * B
        assert same(codes64(kc2), ck2) and same(codes64(vc2), cv2) and same(to64(ks2), sk2) and same(to64(vs2), sv2)
        check_attn("bf16", out2, lse2, q2, K8.values(ck2, sk2, S), K8.values(cv2, sv2, S), (cap2,) * B, k2, v2, L, L, d)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        chain()
    side.synchronize()
    check()
    results = (out1, out2, lse1, lse2, mass, mass2, kc2, vc2)
    first = [x.clone() for x in results]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for x in (kc, kc2, vc2, out1, out2, mass, mass2, lse1, lse2, pos):
        x.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    check()
    for x, y in zip(first, results):
        assert torch.equal(x, y)


def _calls(q, kc, vc, ks, vs, ko, vo, lens, B, Lq, Hq, Hkv, d, P, S, keep, ws):
    """Outputs of the attention, the weights and an eviction, and a function that makes the three calls."""
    out = torch.zeros((B, Lq, Hq * d), dtype=q.dtype, device=DEV)
    lse, mass = torch.zeros((B, Lq, Hq), device=DEV), torch.zeros((B, Hkv, P), device=DEV)
    c2 = [torch.zeros((B, Hkv, keep, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
    s2 = [torch.ones((B, Hkv, cdiv(keep, S)), device=DEV) for _ in range(2)]
    m2 = torch.zeros((B, Hkv, keep), device=DEV)
    pos, l2 = torch.zeros((B, Hkv, keep), dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    dt = bd.BF16 if q.dtype == torch.bfloat16 else bd.F32

    def run(stream=None):
        bd.block_attn_kv8(q, kc, vc, ks, vs, out, B, Lq, Hq, Hkv, d, P, P, S, Lq, dt, prefix_len=lens, k_own=ko, v_own=vo,
                          cap_own=Lq + 3, lse=lse, ws=ws, stream=stream)
        bd.attn_mass_kv8(q, kc, ks, lse, None, mass, B, Lq, Hq, Hkv, d, P, P, S, dt, prefix_len=lens, ws=ws, stream=stream)
        bd.kv8_evict(kc, vc, ks, vs, mass, *c2, *s2, m2, pos, l2, B, Hkv, d, P, P, keep, keep, S, 2, 3, 1, prefix_len=lens,
                     ws=ws, stream=stream)
    return [out, lse, mass, *c2, *s2, m2, pos, l2], run


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_graph_replay_follows_the_device_lengths(dtype, d):
    """Lengths are read when the kernels run: one captured graph serves other lengths, zero among them, and gives the bits
    of direct calls."""
    B, Lq, Hq, Hkv, P, S, keep = 5, 16, 8, 2, 900, 32, 200
    q, kc, vc, ks, vs, _, _, ko, vo = attn_inputs(dtype, B, Lq, Hq, Hkv, d, P, S, None, True, 61)
    lens = torch.full((B,), P, dtype=torch.int32, device=DEV)
    ws = bd.Workspace(64 << 20, DEV)
    outs, run = _calls(q, kc, vc, ks, vs, ko, vo, lens, B, Lq, Hq, Hkv, d, P, S, keep, ws)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for new in ((900, 0, 1, 128, 777), (5, 6, 0, 0, 0), (900, 899, 898, 640, 129)):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        for x in outs:
            x.zero_()
        graph.replay()
        got = [x.clone() for x in outs]
        for x in outs:
            x.zero_()
        run()
        for x, y in zip(got, outs):
            assert torch.equal(x, y)
        assert outs[-1].tolist() == [min(n, keep) for n in new]


def test_two_streams_with_workspaces_of_their_own():
    """Calls that overlap on two streams, each with its own workspace, give the bits they give alone."""
    B, Lq, Hq, Hkv, d, P, S, keep = 4, 32, 16, 4, 128, 2000, 32, 500
    sides, alone = [], []
    for seed in (71, 72):
        q, kc, vc, ks, vs, _, _, ko, vo = attn_inputs("bf16", B, Lq, Hq, Hkv, d, P, S, None, True, seed)
        lens = torch.tensor([P, P - 300 * (seed - 70), 1, 1500], dtype=torch.int32, device=DEV)
        sides.append(_calls(q, kc, vc, ks, vs, ko, vo, lens, B, Lq, Hq, Hkv, d, P, S, keep, bd.Workspace(64 << 20, DEV)))
        sides[-1][1]()
        torch.cuda.synchronize()
        alone.append([x.clone() for x in sides[-1][0]])
    streams = [torch.cuda.Stream() for _ in sides]
    torch.cuda.synchronize()
    for _ in range(20):
        for (outs, run), st in zip(sides, streams):
            run(st)
    torch.cuda.synchronize()
    for (outs, _), want in zip(sides, alone):
        for x, y in zip(outs, want):
            assert torch.equal(x, y)


def test_tensors_off_the_current_device_are_refused():
    x = torch.zeros((1, 1, 16, 128), dtype=torch.bfloat16)
    c = torch.zeros((1, 1, 16, 128), dtype=torch.uint8)
    s = torch.zeros((1, 1, 1))
    with pytest.raises(bd.DllmError) as e:
        bd.kv8_store(x, x, c, c, s, s, 1, 1, 128, 16, 16, 16, 16, bd.BF16)
    assert e.value.code == bd.ERR_INVALID_ARG


def test_long_cache_offsets():
    """More than 2^31 code bytes in one tensor: the last row's keys and values are the ones read, stored and moved."""
    B, Hkv, d, S, cap = 5, 4, 128, 128, 900_000
    free = torch.cuda.mem_get_info()[0]
    assert free > 20 << 30
    kc, vc = torch.zeros((B, Hkv, cap, d), dtype=torch.uint8, device=DEV), torch.zeros((B, Hkv, cap, d), dtype=torch.uint8, device=DEV)
    ks, vs = torch.ones((B, Hkv, cdiv(cap, S)), device=DEV), torch.ones((B, Hkv, cdiv(cap, S)), device=DEV)
    n = 96
    k = rows_like_tokens((B, Hkv, n, d), 51, "k", torch.bfloat16)
    v = rows_like_tokens((B, Hkv, n, d), 51, "v", torch.bfloat16)
    r0 = (cap - n) // S * S
    bd.kv8_store(k, v, kc, vc, ks, vs, B, Hkv, d, n, n, cap, S, bd.BF16, dst_row=r0)
    wc, ws_ = K8.store(to64(k), S)
    assert same(codes64(kc[:, :, r0: r0 + n]), wc) and same(to64(ks[:, :, r0 // S: r0 // S + 1]), ws_)
    # eviction of the last rows, by weight
    P, keep = r0 + n, 64
    mass = torch.zeros((B, Hkv, cap), device=DEV)
    mass[:, :, r0: r0 + keep] = torch.arange(keep, 0, -1, device=DEV).float()
    ko, vo = (torch.zeros((B, Hkv, keep, d), dtype=torch.uint8, device=DEV) for _ in range(2))
    so, to = (torch.zeros((B, Hkv, 1), device=DEV) for _ in range(2))
    mo, kp, lo = torch.zeros((B, Hkv, keep), device=DEV), torch.zeros((B, 1, keep), dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    bd.kv8_evict(kc, vc, ks, vs, mass, ko, vo, so, to, mo, kp, lo, B, Hkv, d, P, cap, keep, keep, S)
    assert torch.equal(kp[:, 0], torch.arange(r0, r0 + keep, dtype=torch.int32, device=DEV).expand(B, keep))
    assert torch.equal(ko, kc[:, :, r0: r0 + keep]) and torch.equal(vo, vc[:, :, r0: r0 + keep])
    # attention over the zero rows and the last ones: their weight from the scores
    q = synth.normal((B, 1, Hkv, d), 1.0, 51, "q", DEV)
    out, lse = torch.empty((B, 1, Hkv * d), dtype=torch.bfloat16, device=DEV), torch.empty((B, 1, Hkv), device=DEV)
    bd.block_attn_kv8(q, kc, vc, ks, vs, out, B, 1, Hkv, Hkv, d, P, cap, S, 1, bd.BF16, lse=lse)
    kv = K8.values(codes64(kc[:, :, r0:P].contiguous()), to64(ks[:, :, r0 // S:]), S)
    vv = K8.values(codes64(vc[:, :, r0:P].contiguous()), to64(vs[:, :, r0 // S:]), S)
    sc = np.einsum("bhd,bhnd->bhn", to64(q)[:, 0], kv) / np.sqrt(d)
    z = np.exp(sc).sum(-1) + r0
    assert np.allclose(to64(lse)[:, 0], np.log(z), atol=1e-4)
    want = np.einsum("bhn,bhnd->bhd", np.exp(sc), vv) / z[..., None]
    tol = 2.0 ** -7 * np.abs(want) + 1e-3 * np.einsum("bhn,bhnd->bhd", np.exp(sc), np.abs(vv)) / z[..., None]
    assert np.all(np.abs(to64(out).reshape(want.shape) - want) <= tol)
    m2 = torch.zeros((B, Hkv, cap), device=DEV)
    bd.attn_mass_kv8(q, kc, ks, lse, None, m2, B, 1, Hkv, Hkv, d, P, cap, S, bd.BF16)
    assert np.allclose(to64(m2[:, :, r0:P]), np.exp(sc) / z[..., None], rtol=1e-3)
    assert not m2[:, :, P:].any()
