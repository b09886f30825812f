"""Cases of the 8-bit KV cache operators: what is measured, in plain torch and through the library.

Four operators that a serving loop calls around one block of a block-diffusion model:

  store  K/V rows into the 8-bit cache: E4M3 codes and one fp32 scale (a power of two) for each run of `S` tokens and
         kv head
  attn   attention of a block's (or one token's, or a prompt chunk's) queries over the 8-bit prefix of each row, of
         its own length, and over the block's own K/V in the storage type; the output and the log-sum-exp
  mass   the weight that those queries put on every cached position, added to an accumulator per kv head
  evict  the cache reduced to the first, the last and the most attended positions, compacted in position order

`run` makes them in elementary torch operations, or, where `own` is true, through the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
MIN_EXP, MAX_EXP = -64, 120    # exponents of the cache's power-of-two scales


# ------------------------------------------------------------------------------------------------------- cases
def _store(name, B, Hkv, d, n, cap, S, dtype="bf16", ragged=0):
    return {"name": name, "op": "store", "B": B, "Hkv": Hkv, "d": d, "n": n, "cap": cap, "S": S, "dtype": dtype,
            "ragged": ragged}


def _attn(name, B, Lq, Hq, Hkv, d, P, S, blk, dtype="bf16", ragged=0):
    return {"name": name, "op": "attn", "B": B, "Lq": Lq, "Hq": Hq, "Hkv": Hkv, "d": d, "P": P, "S": S, "blk": blk,
            "dtype": dtype, "ragged": ragged}


def _mass(name, B, Lq, Hq, Hkv, d, P, S, dtype="bf16", ragged=0):
    return {"name": name, "op": "mass", "B": B, "Lq": Lq, "Hq": Hq, "Hkv": Hkv, "d": d, "P": P, "S": S,
            "dtype": dtype, "ragged": ragged}


def _evict(name, B, Hkv, d, P, S, keep, first, last, per_head=False, ragged=0):
    return {"name": name, "op": "evict", "B": B, "Hkv": Hkv, "d": d, "P": P, "S": S, "keep": keep, "first": first,
            "last": last, "per_head": per_head, "ragged": ragged}


def listed():
    return [
        # a finished 32-token block of 16 rows, each row at its own length: the call after every block
        _store("store-block-16x32", 16, 4, 128, 32, 2720, 32, ragged=640),
        # the prompts of eight thinking-mode rows after their prefill (an odd length)
        _store("store-prompt-8x4091", 8, 4, 128, 4091, 4128, 32),
        # one request: a 32-token block over a 1024-token prefix, where latency counts
        _attn("attn-block-1x1024", 1, 32, 16, 4, 128, 1024, 32, 32),
        # a batch of understanding requests (image and question prefix), lengths of their own
        _attn("attn-block-16x2688", 16, 32, 16, 4, 128, 2688, 32, 32, ragged=640),
        # long reasoning prefixes: the largest read of the cache
        _attn("attn-block-8x32768", 8, 32, 16, 4, 128, 32768, 64, 32),
        # single tokens of many rows (block length 1), seven query heads to a kv head, odd ragged lengths
        _attn("attn-token-64x4001", 64, 1, 28, 4, 128, 4001, 16, 1, ragged=3001),
        # a chunk of a long prompt, block-causal inside the chunk, over the part that is cached already
        _attn("attn-chunk-2x500-4000", 2, 500, 16, 4, 128, 4000, 128, 32),
        # the small fp32 model: four heads of 64
        _attn("attn-fp32-3x300", 3, 16, 4, 4, 64, 300, 16, 16, dtype="f32", ragged=171),
        # the weights that the understanding batch's block puts on its prefixes
        _mass("mass-block-16x2688", 16, 32, 16, 4, 128, 2688, 32, ragged=640),
        # the same over long prefixes
        _mass("mass-block-4x32768", 4, 32, 16, 4, 128, 32768, 64),
        # thinking mode, half of every prefix kept, one set of positions for all heads
        _evict("evict-8x4096", 8, 4, 128, 4096, 32, 2048, 4, 128),
        # one very long context, an eighth kept, a set of its own for every kv head
        _evict("evict-heads-1x131072", 1, 4, 128, 131072, 16, 16384, 4, 512, per_head=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "attn", "attn", "mass", "evict"])
    S = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    f32 = op != "evict" and rng.random() < 0.2
    d = rng.choice([32, 64, 80, 128]) if f32 else 128
    B = _log_int(rng, 1, 64)
    if op == "store":
        n = _log_int(rng, 1, max(2, min(8192, (1 << 24) // (B * Hkv * d))))
        c = _store("", B, Hkv, d, n, n + rng.randint(0, 700), S, "f32" if f32 else "bf16")
        c["ragged"] = rng.choice([0, c["cap"] - n])
    elif op in ("attn", "mass"):
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        Lq = rng.choice([1, 1, 2, 7, 16, 31, 32, 32, 64, 129, 300])
        if f32:
            B, Lq = min(B, 4), min(Lq, 32)
        room = (1 << 23) // (B * Hkv) if not f32 else 1 << 11
        P = _log_int(rng, 1, max(2, min(65536, room // max(1, G * Lq // 128))))
        ragged = rng.choice([0, P // 2, P])
        if op == "attn":
            c = _attn("", B, Lq, G * Hkv, Hkv, d, P, S, rng.choice([1, 16, 32, 4096]), "f32" if f32 else "bf16", ragged)
        else:
            c = _mass("", B, Lq, G * Hkv, Hkv, d, P, S, "f32" if f32 else "bf16", ragged)
    else:
        P = _log_int(rng, 2, max(4, min(131072, (1 << 19) // (B * Hkv))))
        keep = rng.randint(1, P)
        first = rng.randint(0, min(8, keep))
        c = _evict("", B, Hkv, rng.choice([64, 128]), P, S, keep, first, rng.randint(0, (keep - first) // 2),
                   rng.random() < 0.5, rng.choice([0, P // 2, P]))
    del c["name"]
    return c


def _lengths(case, most):
    """The rows' lengths, from the case alone: most, or spread over [most - ragged, most]."""
    r, B = case["ragged"], case["B"]
    return [most - (i * 7919 + 1) * 31 % (r + 1) if r else most for i in range(B)]


def _dst_rows(case):
    """Where each row's stored tokens go: whole scale runs, inside the cache."""
    room = (case["cap"] - case["n"]) // case["S"]
    return [((case["cap"] - case["n"] - x) // case["S"] if case["ragged"] else room) * case["S"]
            for x in [min(case["cap"] - case["n"], y) for y in [(i * 7919 + 1) * 31 % (case["ragged"] + 1)
                                                               for i in range(case["B"])]]]


def _dt(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def work(case):
    B, Hkv, d, S = case["B"], case["Hkv"], case["d"], case["S"]
    es = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if case["op"] == "store":
        rows = B * Hkv * case["n"]
        return {"bytes": 2 * (rows * d * (es + 1) + rows / S * 4), "flops": 2.0 * rows * d}
    if case["op"] in ("attn", "mass"):
        keys, Lq, Hq = sum(_lengths(case, case["P"])), case["Lq"], case["Hq"]
        cached = keys * Hkv * (d + 4 / S)
        if case["op"] == "mass":
            return {"bytes": cached + B * Lq * Hq * (d * es + 4) + 2 * keys * Hkv * 4,
                    "flops": 2.0 * keys * Lq * Hq * d}
        blk = case["blk"]
        seen = sum(min(Lq, (i // blk + 1) * blk) for i in range(Lq))     # own keys over the queries of one row
        return {"bytes": 2 * cached + B * Lq * d * es * (2 * Hq + 2 * Hkv) + B * Lq * Hq * 4,
                "flops": 4.0 * d * Hq * (keys * Lq + B * seen)}
    lens = _lengths(case, case["P"])
    kept = sum(min(x, case["keep"]) for x in lens) * Hkv
    return {"bytes": sum(lens) * Hkv * 4 + kept * (4 * d + 4 + 16 / S), "flops": 2.0 * kept * d + sum(lens) * Hkv}


# ------------------------------------------------------------------------------------------------- plain pieces
def _runs(x, S):
    """[..., n, d] in runs of S tokens, the last filled up with zeros: [..., ceil(n / S), S, d]."""
    n = x.shape[-2]
    m = -(-n // S)
    if m * S != n:
        x = torch.cat([x, x.new_zeros(*x.shape[:-2], m * S - n, x.shape[-1])], -2)
    return x.reshape(*x.shape[:-2], m, S, x.shape[-1])


def _quantise(x, S):
    """Codes [..., n, d] (E4M3) and scales [..., ceil(n / S)] of x: the smallest power of two that brings the run's
    largest magnitude to at most 448 (= 0.875 * 2^9)."""
    n = x.shape[-2]
    r = _runs(x.float(), S)
    m, e = torch.frexp(r.abs().amax((-2, -1)))
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(MIN_EXP, MAX_EXP)
    k = torch.where(m == 0, MIN_EXP, k)
    scale = torch.ldexp(torch.ones_like(m), k)
    codes = (r * torch.ldexp(torch.ones_like(m), -k)[..., None, None]).to(E4M3)
    return codes.reshape(*x.shape[:-2], -1, x.shape[-1])[..., :n, :], scale


def _values(codes, scale, S):
    """What the codes [..., n, d] stand for, in 32 bits."""
    n = codes.shape[-2]
    return codes.float() * scale.repeat_interleave(S, -1)[..., :n, None]


def _gen(seed, k):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 16 + k)
    return g


def _tokens(shape, g):
    """K or V rows: normal values, the rows' sizes varying as tokens' do."""
    x = torch.randn(shape, generator=g, device=DEV)
    return x * torch.exp(0.3 * torch.randn((*shape[:-1], 1), generator=g, device=DEV))


# ----------------------------------------------------------------------------------------------------- prepare
def prepare(case, seed):
    op, B, Hkv, d, S = case["op"], case["B"], case["Hkv"], case["d"], case["S"]
    s = {"case": dict(case)}
    if op == "store":
        n, cap = case["n"], case["cap"]
        s["k"] = _tokens((B, Hkv, n, d), _gen(seed, 0)).to(_dt(case))
        s["v"] = _tokens((B, Hkv, n, d), _gen(seed, 1)).to(_dt(case))
        s["rows"] = torch.tensor(_dst_rows(case), dtype=torch.int32, device=DEV)
        for x in ("k", "v"):
            s[x + "_codes"] = torch.zeros((B, Hkv, cap, d), dtype=torch.uint8, device=DEV).view(E4M3)
            s[x + "_scale"] = torch.ones((B, Hkv, -(-cap // S)), device=DEV)
        return s
    P = case["P"]
    for i, x in enumerate(("k", "v")):
        if op == "mass" and x == "v":
            continue
        parts = [_quantise(_tokens((Hkv, P, d), _gen(seed * 1024 + b, i)), S) for b in range(B)]
        s[x + "_codes"] = torch.stack([p[0].view(torch.uint8) for p in parts]).view(E4M3)
        s[x + "_scale"] = torch.stack([p[1] for p in parts])
    s["lens"] = torch.tensor(_lengths(case, P), dtype=torch.int32, device=DEV)
    if op == "evict":
        keep, per = case["keep"], case["per_head"]
        # accumulated weights: heavy-tailed, a few positions with most of the weight
        s["mass"] = torch.exp(2.0 * torch.randn((B, Hkv, P), generator=_gen(seed, 5), device=DEV))
        for x in ("k", "v"):
            s[x + "_out"] = torch.zeros((B, Hkv, keep, d), dtype=torch.uint8, device=DEV).view(E4M3)
            s[x + "_scale_out"] = torch.ones((B, Hkv, -(-keep // S)), device=DEV)
        s["mass_out"] = torch.zeros((B, Hkv, keep), device=DEV)
        s["keep_pos"] = torch.full((B, Hkv if per else 1, keep), -1, dtype=torch.int32, device=DEV)
        s["len_out"] = torch.zeros((B,), dtype=torch.int32, device=DEV)
        return s
    Lq, Hq = case["Lq"], case["Hq"]
    s["q"] = (1.5 * torch.randn((B, Lq, Hq, d), generator=_gen(seed, 2), device=DEV)).to(_dt(case))
    s["lse"] = torch.zeros((B, Lq, Hq), device=DEV)
    if op == "attn":
        s["k_own"] = _tokens((B, Hkv, Lq, d), _gen(seed, 3)).to(_dt(case))
        s["v_own"] = _tokens((B, Hkv, Lq, d), _gen(seed, 4)).to(_dt(case))
        s["out"] = torch.zeros((B, Lq, Hq * d), dtype=_dt(case), device=DEV)
    else:
        # the log-sum-exp that the attention left: over the prefix here, plus what the block's own keys added
        for b in range(B):
            k = _values(s["k_codes"][b], s["k_scale"][b], S)[:, : _lengths(case, P)[b]]
            sc = torch.einsum("lhgd,hpd->lhgp", s["q"][b].float().reshape(Lq, Hkv, Hq // Hkv, d), k) / math.sqrt(d)
            s["lse"][b] = torch.logaddexp(torch.logsumexp(sc, -1), torch.tensor(2.0, device=DEV)).reshape(Lq, Hq)
        s["mass"] = torch.rand((B, Hkv, P), generator=_gen(seed, 6), device=DEV)
        s["mass_out"] = torch.zeros((B, Hkv, P), device=DEV)
    return s


# ------------------------------------------------------------------------------------------------- plain forms
def _plain_store(s):
    c = s["case"]
    S, n = c["S"], c["n"]
    at = torch.arange(n, device=DEV) + s["rows"].long()[:, None]                  # [B, n]
    runs = torch.arange(-(-n // S), device=DEV) + s["rows"].long()[:, None] // S
    out = {}
    for x in ("k", "v"):
        codes, scale = _quantise(s[x], S)
        idx = at[:, None, :, None].expand(codes.shape)
        s[x + "_codes"].view(torch.uint8).scatter_(2, idx, codes.contiguous().view(torch.uint8))
        s[x + "_scale"].scatter_(2, runs[:, None].expand(scale.shape), scale)
        out[x], out[x + "_scale"] = s[x + "_codes"], s[x + "_scale"]
    return out


def _scores(s):
    """softmax logits over the prefix [B, Hkv, Lq * G, P] (rows: query, then head of the group), -inf past a row's
    length, in 32 bits."""
    c = s["case"]
    B, Lq, Hkv, d, P = c["B"], c["Lq"], c["Hkv"], c["d"], c["P"]
    G = c["Hq"] // Hkv
    q = s["q"].float().reshape(B, Lq, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Lq * G, d)
    sc = q @ _values(s["k_codes"], s["k_scale"], c["S"]).transpose(-1, -2) / math.sqrt(d)
    hidden = torch.arange(P, device=DEV) >= s["lens"][:, None, None, None]
    return q, sc.masked_fill_(hidden, -math.inf)


def _plain_attn(s):
    c = s["case"]
    B, Lq, Hkv, d, P, blk = c["B"], c["Lq"], c["Hkv"], c["d"], c["P"], c["blk"]
    G = c["Hq"] // Hkv
    q, sc = _scores(s)
    i = torch.arange(Lq, device=DEV) // blk
    own_sc = q @ s["k_own"].float().transpose(-1, -2) / math.sqrt(d)
    own_sc.masked_fill_((i[None, :] > i[:, None]).repeat_interleave(G, 0), -math.inf)
    sc = torch.cat([sc, own_sc], -1)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    o = (p[..., :P] @ _values(s["v_codes"], s["v_scale"], c["S"]) + p[..., P:] @ s["v_own"].float()) / l
    lse = (m + torch.log(l)).squeeze(-1)

    def rows(x):
        return x.reshape(B, Hkv, Lq, G, -1).permute(0, 2, 1, 3, 4)

    return {"out": rows(o).reshape(B, Lq, -1).to(s["q"].dtype), "lse": rows(lse).reshape(B, Lq, -1)}


def _plain_mass(s):
    c = s["case"]
    B, Lq, Hkv, P = c["B"], c["Lq"], c["Hkv"], c["P"]
    lse = s["lse"].reshape(B, Lq, Hkv, -1).permute(0, 2, 1, 3).reshape(B, Hkv, -1, 1)
    add = torch.exp(_scores(s)[1] - lse).sum(-2)
    seen = torch.arange(P, device=DEV) < s["lens"][:, None, None]
    return {"mass": torch.where(seen, s["mass"] + add, s["mass_out"])}


def _plain_evict(s):
    c = s["case"]
    B, Hkv, d, P, S, keep = c["B"], c["Hkv"], c["d"], c["P"], c["S"], c["keep"]
    j = torch.arange(P, device=DEV)
    key = s["mass"].double() if c["per_head"] else s["mass"].double().sum(1, keepdim=True)
    key = key.float()                                                            # [B, Hkv or 1, P]
    lens = s["lens"].long()[:, None, None]
    key = torch.where((j < c["first"]) | (j >= lens - c["last"]), math.inf, key)
    key = torch.where(j < lens, key, -1.0)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    count = torch.clamp(lens, max=keep)
    t = torch.arange(keep, device=DEV)
    pos = torch.where(t < count, order, P).sort(-1).values                       # ascending, the kept ones first
    live = (t < count).expand(pos.shape)
    at = torch.where(live, pos, 0).expand(B, Hkv, keep)
    live_h = live.expand(B, Hkv, keep)
    out = {"keep_pos": torch.where(live, pos, -1).to(torch.int32), "len": count.reshape(B).to(torch.int32),
           "mass": torch.where(live_h, s["mass"].gather(-1, at), 0.0)}
    for x in ("k", "v"):
        old = torch.where(live_h, s[x + "_scale"].gather(-1, at // S), 0.0)       # [B, Hkv, keep]
        new = _runs(old[..., None], S).amax((-2, -1))                             # [B, Hkv, runs]
        out[x + "_scale"] = torch.where(new > 0, new, 1.0)
        ratio = old / out[x + "_scale"].repeat_interleave(S, -1)[..., :keep]
        codes = s[x + "_codes"].view(torch.uint8).gather(2, at[..., None].expand(B, Hkv, keep, d)).view(E4M3)
        out[x] = torch.where(live_h[..., None], codes.float() * ratio[..., None], 0.0).to(E4M3)
    return out


# ------------------------------------------------------------------------------------------ the library's calls
_ws = None    # one workspace for all calls, as a serving loop keeps it


def _workspace(bd):
    global _ws
    if _ws is None:
        _ws = bd.Workspace(64 << 20, DEV)
    return _ws


def _own_run(s):
    from block_diffusion_moe_dllm_b200 import binding as bd
    c = s["case"]
    dtype = bd.BF16 if c.get("dtype", "bf16") == "bf16" else bd.F32
    B, Hkv, d, S = c["B"], c["Hkv"], c["d"], c["S"]
    if c["op"] == "store":
        bd.kv8_store(s["k"], s["v"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], B, Hkv, d, c["n"],
                     c["n"], c["cap"], S, dtype, dst_rows=s["rows"])
        return {"k": s["k_codes"], "v": s["v_codes"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if c["op"] == "attn":
        bd.block_attn_kv8(s["q"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["out"], B, c["Lq"],
                          c["Hq"], Hkv, d, c["P"], c["P"], S, c["blk"], dtype, prefix_len=s["lens"],
                          k_own=s["k_own"], v_own=s["v_own"], cap_own=c["Lq"], lse=s["lse"], ws=_workspace(bd))
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "mass":
        bd.attn_mass_kv8(s["q"], s["k_codes"], s["k_scale"], s["lse"], s["mass"], s["mass_out"], B, c["Lq"], c["Hq"],
                         Hkv, d, c["P"], c["P"], S, dtype, prefix_len=s["lens"], ws=_workspace(bd))
        return {"mass": s["mass_out"]}
    bd.kv8_evict(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["mass"], s["k_out"], s["v_out"],
                 s["k_scale_out"], s["v_scale_out"], s["mass_out"], s["keep_pos"], s["len_out"], B, Hkv, d, c["P"],
                 c["P"], c["keep"], c["keep"], S, n_first=c["first"], n_last=c["last"], per_head=int(c["per_head"]),
                 prefix_len=s["lens"], ws=_workspace(bd))
    return {"keep_pos": s["keep_pos"], "len": s["len_out"], "mass": s["mass_out"], "k": s["k_out"], "v": s["v_out"],
            "k_scale": s["k_scale_out"], "v_scale": s["v_scale_out"]}


_PLAIN = {"store": _plain_store, "attn": _plain_attn, "mass": _plain_mass, "evict": _plain_evict}


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------------- exact
def _e4m3_64(x):
    """x in 64 bits rounded to the nearest E4M3 value, ties to even, by the format's definition."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e - 1, min=-6) - 3)
    return torch.clamp(torch.round(x / step) * step, -448.0, 448.0)


def _scale_64(amax):
    """2^k, k the least integer with amax <= 448 * 2^k, within the exponents' limits."""
    k = torch.ceil(torch.log2(torch.clamp(amax, min=1e-300) / 448.0))
    k = torch.where(amax > 448.0 * torch.exp2(k), k + 1, k)
    k = torch.where(amax <= 448.0 * torch.exp2(k - 1), k - 1, k)
    return torch.exp2(torch.clamp(k, MIN_EXP, MAX_EXP))


def _row_values_64(s, x, b, h, n):
    sc = s[x + "_scale"][b, h].double()[torch.arange(n, device=DEV) // s["case"]["S"]]
    return s[x + "_codes"][b, h, :n].double() * sc[:, None]


def _exact_store(s):
    c = s["case"]
    S, n = c["S"], c["n"]
    out = {}
    for x in ("k", "v"):
        codes, scale = s[x + "_codes"].double(), s[x + "_scale"].double()
        for b, r0 in enumerate(_dst_rows(c)):
            for t in range(0, n, S):
                part = s[x][b, :, t: t + S].double()
                sc = _scale_64(part.abs().amax((1, 2)))
                codes[b, :, r0 + t: r0 + t + part.shape[1]] = _e4m3_64(part / sc[:, None, None])
                scale[b, :, (r0 + t) // S] = sc
        out[x], out[x + "_scale"] = codes, scale
    return out


def _exact_attn(s):
    c = s["case"]
    B, Lq, Hq, Hkv, d, blk = c["B"], c["Lq"], c["Hq"], c["Hkv"], c["d"], c["blk"]
    G = Hq // Hkv
    out = torch.zeros((B, Lq, Hq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, Lq, Hq), dtype=torch.float64, device=DEV)
    i = torch.arange(Lq, device=DEV) // blk
    for b, n in enumerate(_lengths(c, c["P"])):
        for h in range(Hkv):
            k = torch.cat([_row_values_64(s, "k", b, h, n), s["k_own"][b, h].double()])
            v = torch.cat([_row_values_64(s, "v", b, h, n), s["v_own"][b, h].double()])
            seen = torch.cat([torch.ones((Lq, n), dtype=torch.bool, device=DEV), i[None, :] <= i[:, None]], 1)
            for g in range(h * G, h * G + G):
                z = torch.where(seen, s["q"][b, :, g].double() @ k.T / math.sqrt(d), -math.inf)
                lse[b, :, g] = torch.logsumexp(z, 1)
                out[b, :, g] = torch.softmax(z, 1) @ v
    return {"out": out.reshape(B, Lq, Hq * d), "lse": lse}


def _exact_mass(s):
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    mass = s["mass_out"].double()
    for b, n in enumerate(_lengths(c, c["P"])):
        for h in range(c["Hkv"]):
            k = _row_values_64(s, "k", b, h, n)
            mass[b, h, :n] = s["mass"][b, h, :n].double()
            for g in range(h * G, h * G + G):
                z = s["q"][b, :, g].double() @ k.T / math.sqrt(c["d"])
                mass[b, h, :n] += torch.exp(z - s["lse"][b, :, g, None].double()).sum(0)
    return {"mass": mass}


def _exact_evict(s):
    c = s["case"]
    B, Hkv, S, keep, per = c["B"], c["Hkv"], c["S"], c["keep"], c["per_head"]
    mass = s["mass"].double().cpu().numpy()
    pos = np.full((B, Hkv if per else 1, keep), -1, dtype=np.int32)
    lens = _lengths(c, c["P"])
    out = {x + "_scale": torch.ones((B, Hkv, -(-keep // S)), dtype=torch.float64, device=DEV) for x in ("k", "v")}
    out |= {x: torch.zeros((B, Hkv, keep, c["d"]), dtype=torch.float64, device=DEV) for x in ("k", "v")}
    out["mass"] = torch.zeros((B, Hkv, keep), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        for w in range(pos.shape[1]):
            total = (mass[b, w, :n] if per else mass[b, :, :n].sum(0)).astype(np.float32)
            must = np.zeros(n, dtype=bool)
            must[: c["first"]] = True
            must[max(0, n - c["last"]):] = True
            chosen = np.lexsort((np.arange(n), -total, ~must))[:keep]
            pos[b, w, : len(chosen)] = np.sort(chosen)
        for h in range(Hkv):
            at = torch.from_numpy(pos[b, h if per else 0, : min(n, keep)].astype(np.int64)).to(DEV)
            out["mass"][b, h, : len(at)] = s["mass"][b, h, at].double()
            for x in ("k", "v"):
                old = s[x + "_scale"][b, h, at // S].double()
                run_of = torch.arange(len(at), device=DEV) // S
                new = out[x + "_scale"][b, h]
                if len(at):
                    top = torch.zeros_like(new).scatter_reduce(0, run_of, old, "amax")
                    new.copy_(torch.where(top > 0, top, new))
                out[x][b, h, : len(at)] = _e4m3_64(s[x + "_codes"][b, h, at].double() * (old / new[run_of])[:, None])
    return out | {"keep_pos": torch.from_numpy(pos).to(DEV),
                  "len": torch.tensor([min(n, keep) for n in lens], dtype=torch.int32, device=DEV)}


def exact(case, seed):
    return {"store": _exact_store, "attn": _exact_attn, "mass": _exact_mass,
            "evict": _exact_evict}[case["op"]](prepare(case, seed))
