"""The 8-bit KV cache's calls on parts of longer arrays and on rows of lengths of their own (GPU). Each gives the bits it
gives on a copy of the part, or on the row alone."""
import pytest
import torch

from block_diffusion_moe_dllm_b200 import binding as bd
from block_diffusion_moe_dllm_b200 import synth
from test_gpu_kv8 import DEV, DT, cdiv, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bd.load()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("B,Hkv,cap,r0,S", [(1, 1, 200, 64, 32), (2, 3, 333, 48, 16), (1, 2, 129, 128, 128)])
def test_attention_and_weights_of_a_part(dtype, d, B, Hkv, cap, r0, S):
    """Rows [r0, cap) of every head: the last head's rows end where the memory ends."""
    Lq, Hq, P = 3, 2 * Hkv, cap - r0
    kc, vc, ks, vs, _, _ = make_cache(B, Hkv, cap, d, S, 101)
    q = synth.normal((B, Lq, Hq, d), 1.5, 101, "q", DEV, synth.torch_dtype(dtype))
    got = []
    for part in (True, False):
        c = [x[:, :, r0:] if part else x[:, :, r0:].contiguous() for x in (kc, vc)]
        s = [x[:, :, r0 // S:] if part else x[:, :, r0 // S:].contiguous() for x in (ks, vs)]
        stride = cap if part else P
        out = torch.full((B, Lq, Hq * d), float("nan"), dtype=q.dtype, device=DEV)
        lse = torch.full((B, Lq, Hq), float("nan"), device=DEV)
        bd.block_attn_kv8(q, *c, *s, out, B, Lq, Hq, Hkv, d, P, stride, S, 1, DT[dtype], lse=lse)
        mass = torch.full((B, Hkv, stride), 3.0, device=DEV)
        bd.attn_mass_kv8(q, c[0], s[0], lse, None, mass, B, Lq, Hq, Hkv, d, P, stride, S, DT[dtype])
        assert torch.all(mass[:, :, P:] == 3.0)
        got.append((out, lse, mass[:, :, :P]))
    assert all(torch.equal(x, y) for x, y in zip(*got)) and torch.isfinite(got[0][0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ragged_rows_stored_in_one_call(dtype):
    """Rows of lengths of their own by a position list that is -1 past each end: what lies there leaves no trace, each row
    is stored as it is alone, and the next block goes behind a row whose length is a multiple of the run."""
    B, Hkv, d, n, S, cap = 3, 2, 64, 200, 32, 256
    lens = (77, 200, 96)
    t = synth.torch_dtype(dtype)
    k, v = (synth.normal((B, Hkv, n, d), 1.0, 102, x, DEV, t) for x in ("k", "v"))
    for b, m in enumerate(lens):
        k[b, :, m:], v[b, :, m:] = 1e30, float("nan")
    pos = torch.arange(n, dtype=torch.int32, device=DEV).repeat(B, 1)
    pos = torch.where(pos < torch.tensor(lens, device=DEV)[:, None], pos, -1)

    def empty(rows):
        return ([torch.zeros((rows, Hkv, cap, d), dtype=torch.uint8, device=DEV) for _ in range(2)],
                [torch.zeros((rows, Hkv, cap // S), device=DEV) for _ in range(2)])

    codes, scale = empty(B)
    bd.kv8_store(k, v, *codes, *scale, B, Hkv, d, n, n, cap, S, DT[dtype], src_pos=pos)
    for b, m in enumerate(lens):
        c1, s1 = empty(1)
        bd.kv8_store(k[b: b + 1], v[b: b + 1], *c1, *s1, 1, Hkv, d, m, n, cap, S, DT[dtype])
        for x, y in zip(codes + scale, c1 + s1):
            rows = m if x.dtype == torch.uint8 else cdiv(m, S)
            assert torch.equal(x[b, :, :rows], y[0, :, :rows])
            assert x.dtype != torch.uint8 or not x[b, :, m:n].any()
    # of the three lengths only 96 starts a run: the others are left as they were
    before = [x.clone() for x in codes + scale]
    blk = [synth.normal((B, Hkv, 32, d), 1.0, 103, x, DEV, t) for x in ("k", "v")]
    bd.kv8_store(*blk, *codes, *scale, B, Hkv, d, 32, 32, cap, S, DT[dtype],
                 dst_rows=torch.tensor(lens, dtype=torch.int32, device=DEV))
    for x, y in zip(codes + scale, before):
        assert torch.equal(x[:2], y[:2]) and not torch.equal(x[2], y[2])


def test_fewer_tiles_than_ctas():
    """Device lengths far below P: most CTAs of the launch have no share of the tiles, with several heads to a row. The
    results are those of a call whose P says so: the same bits for the weights, and for the outputs one rounding (bf16's
    step is at most 2^-7 of the value) of sums that were split elsewhere."""
    B, Lq, Hq, Hkv, d, P, S = 3, 5, 8, 4, 128, 8192, 64
    lens = torch.tensor([1, 0, 130], dtype=torch.int32, device=DEV)
    kc, vc, ks, vs, _, _ = make_cache(B, Hkv, P, d, S, 104)
    q = synth.normal((B, Lq, Hq, d), 1.5, 104, "q", DEV, torch.bfloat16)
    want = None
    for most in (130, P):
        out = torch.full((B, Lq, Hq * d), float("nan"), dtype=torch.bfloat16, device=DEV)
        lse = torch.full((B, Lq, Hq), float("nan"), device=DEV)
        mass = torch.full((B, Hkv, P), 2.0, device=DEV)
        bd.block_attn_kv8(q, kc, vc, ks, vs, out, B, Lq, Hq, Hkv, d, most, P, S, 1, bd.BF16, prefix_len=lens, lse=lse)
        bd.attn_mass_kv8(q, kc, ks, lse, None, mass, B, Lq, Hq, Hkv, d, most, P, S, bd.BF16, prefix_len=lens)
        want = want or (out, lse, mass)
    assert torch.equal(mass, want[2]) and torch.equal(lse[1], want[1][1])
    assert torch.allclose(out.float(), want[0].float(), rtol=2 ** -7, atol=1e-5) and not out[1].any()
    assert torch.allclose(lse[::2], want[1][::2], rtol=1e-6, atol=1e-6)
