"""The measured cases of the position and 4-bit cache operators: rotary positions, the cache writers that rotate on
the way, the attention over 4-bit latent rows, and the reader of cached rows.

Plain forms (``own`` false) are elementary torch operations in 32 bits (angles in 64); with ``own`` true ``run`` makes
the calls a user makes of ``dsa_indexed_sparse_gb300``.  The sizes are those of the decode and prefill configurations
of this repository: 128 heads over 512 latent + 64 rope dims, 64-token pages, 2048 selected rows.
"""
import math

import torch

own = False

D_LATENT, D_ROPE, HEADS, PAGE = 512, 64, 128, 64
D_ROW = D_LATENT + D_ROPE
E2M1_ROW, FP8_ROW = 432, 656
DEV = "cuda" if torch.cuda.is_available() else "cpu"
E2M1_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode token's 128 rope heads, projected apart and rotated into the attention query
        dict(name="rope decode 1", op="rope", T=1, H=128, d=64, dtype="bf16", layout="interleaved", scaling="none",
             inverse=False, ctx=32768, out_row=576),
        # a whole prompt's rope heads, YaRN-scaled positions
        dict(name="rope prompt 16384", op="rope", T=16384, H=128, d=64, dtype="bf16", layout="interleaved",
             scaling="yarn", inverse=False, ctx=131072, out_row=576),
        # the inverse (the gradient) on fp32 indexer heads, half layout, the first 64 of 128 dims, an odd count of
        # tokens at positions up to a million
        dict(name="rope inverse f32 half", op="rope", T=333, H=64, d=64, dtype="f32", layout="half", scaling="ntk",
             inverse=True, ctx=1 << 20, out_row=128),
        # the new tokens of a decode batch into the 4-bit cache, read back as the values they stand for
        dict(name="append 4-bit decode 64", op="append", fmt="e2m1", T=64, B=64, ctx=8192, scaling="yarn"),
        # a prompt chunk into the bf16 cache (the whole pool comes back)
        dict(name="append bf16 chunk 8192", op="append", fmt="bf16", T=8192, B=1, ctx=16384, scaling="none"),
        # an odd chunk of seven sequences into FP8 rows, read back
        dict(name="append fp8 chunk 1001", op="append", fmt="e4m3", T=1001, B=7, ctx=4000, scaling="linear"),
        # one decode token over a 32768-token cache: the smallest call
        dict(name="attention decode 1", op="attention", T=1, B=1, ctx=32768, K=2048, holes=False),
        # a decode batch over caches of up to 8192 tokens
        dict(name="attention decode 64", op="attention", T=64, B=64, ctx=8192, K=2048, holes=False),
        # an odd batch with an odd selection, unused entries in the middle and a row that selects nothing
        dict(name="attention ragged 7x777", op="attention", T=7, B=7, ctx=3001, K=777, holes=True),
        # a causal prompt chunk: 2048 queries at the end of a 4096-token sequence
        dict(name="attention chunk 2048", op="attention", T=2048, B=1, ctx=4096, K=2048, holes=False),
        # a cached prefix expanded to bf16 again
        dict(name="read 4-bit 65536", op="read", fmt="e2m1", T=65536, B=4, ctx=16384, dtype="bf16"),
        # a short odd prefix of tile-scaled FP8 rows to fp32
        dict(name="read fp8 tiles 333", op="read", fmt="e4m3_t128", T=333, B=3, ctx=777, dtype="f32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "read"])
    if op == "rope":
        H, d, dtype = rng.choice([1, 16, 32, 64, 128]), rng.choice([32, 64, 128]), rng.choice(["bf16", "f32"])
        most = 16384 * 128 * 64 // (max(H, 32) * d * (1 if dtype == "bf16" else 2))
        return dict(op=op, T=_spread(rng, 1, most), H=H, d=d, dtype=dtype,
                    layout=rng.choice(["interleaved", "half"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    inverse=rng.random() < 0.3, ctx=_spread(rng, 64, 1 << 20), out_row=rng.choice([0, 576]))
    if op == "append":
        B = _spread(rng, 1, 64)
        per = _spread(rng, 1, max(1, 8192 // B))
        return dict(op=op, fmt=rng.choice(["bf16", "f32", "e4m3", "e4m3_t128", "e2m1"]), T=B * per, B=B,
                    ctx=per + _spread(rng, 1, max(1, 16384 // B)), scaling=rng.choice(["none", "linear", "ntk", "yarn"]))
    if op == "attention":
        B = _spread(rng, 1, 64)
        per = 1 if rng.random() < 0.5 else _spread(rng, 1, max(1, 1024 // B))
        ctx = per + _spread(rng, 16, 131072 // B)
        return dict(op=op, T=B * per, B=B, ctx=ctx, K=_spread(rng, 1, 2048), holes=rng.random() < 0.5)
    B = _spread(rng, 1, 16)
    ctx = _spread(rng, 1, 65536 // B)
    return dict(op=op, fmt=rng.choice(["bf16", "f32", "e4m3", "e4m3_t128", "e2m1"]), T=B * ctx, B=B, ctx=ctx,
                dtype=rng.choice(["bf16", "f32"]))


def _selected(case):
    """Rows that the queries of an attention case may select, holes not counted."""
    per = case["T"] // case["B"]
    return case["B"] * sum(min(case["K"], case["ctx"] - per + i + 1) for i in range(per))


def _row_bytes(fmt):
    return {"bf16": 2 * D_ROW, "f32": 4 * D_ROW, "e4m3": FP8_ROW, "e4m3_t128": FP8_ROW, "e2m1": E2M1_ROW}[fmt]


def work(case):
    T = case["T"]
    if case["op"] == "rope":
        n = T * case["H"] * case["d"]
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4) + 4 * T, "flops": 3 * n}
    if case["op"] == "append":
        fmt = case["fmt"]
        src = D_ROW * (4 if fmt == "f32" else 2)
        back = 0 if fmt in ("bf16", "f32") else D_ROW * 2
        return {"bytes": T * (src + _row_bytes(fmt) + back + 8), "flops": T * (3 * D_ROPE + 4 * D_LATENT)}
    if case["op"] == "attention":
        rows = _selected(case)
        distinct = min(rows, case["B"] * case["ctx"])
        return {"bytes": distinct * E2M1_ROW + T * (HEADS * (D_ROW * 2 + D_LATENT * 2 + 4) + case["K"] * 4),
                "flops": 2 * HEADS * (D_ROW + D_LATENT) * rows}
    return {"bytes": T * (_row_bytes(case["fmt"]) + D_ROW * (2 if case["dtype"] == "bf16" else 4) + 8),
            "flops": T * D_LATENT}


# ------------------------------------------------------------------------------------------------- the formats

def _frequencies(d, scaling):
    """Angular frequencies [d/2] in 64 bits and the factor on cos and sin."""
    theta, factor, original = 10000.0, 32.0, 4096.0
    if scaling == "ntk":
        theta = theta * factor ** (d / (d - 2.0))
    f = theta ** (-torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        turns = [d * math.log(original / (b * 2.0 * math.pi)) / (2.0 * math.log(theta)) for b in (32.0, 1.0)]
        lo, hi = max(math.floor(turns[0]), 0), min(math.ceil(turns[1]), d - 1)
        ramp = ((torch.arange(d // 2, dtype=torch.float64, device=DEV) - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return f * (1.0 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _rotate(x, pos, freq, factor, layout, inverse):
    """x [T, ..., d] in 32 bits, rotated by the angles pos * freq (64 bits)."""
    angle = pos.double()[:, None] * freq[None, :]
    cos, sin = (factor * angle.cos()).float(), (factor * angle.sin()).float()
    if x.dim() == 3:
        cos, sin = cos[:, None, :], sin[:, None, :]
    if inverse:
        sin = -sin
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if layout == "interleaved" else (x[..., :half], x[..., half:])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack([u, v], dim=-1).flatten(-2) if layout == "interleaved" else torch.cat([u, v], dim=-1)


def _power_of_two_below(amax, bias):
    """Exponent floor(log2 amax) - bias of positive numbers."""
    return torch.frexp(amax)[1] - 1 - bias


def _e2m1_codes(x, scale):
    """The 4-bit codes nearest to x / scale (ties to the even code), 0 where the scale is 0."""
    q = torch.where(scale > 0, x / torch.where(scale > 0, scale, torch.ones_like(scale)), torch.zeros_like(x))
    a = q.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() +
            (a >= 3.5).int() + (a > 5.0).int())
    return code + 8 * torch.signbit(q).int()


def _encode(latent, fmt):
    """Latent rows [n, 512] (32-bit values) as a quantised row's bytes before its rope part."""
    n = latent.shape[0]
    if fmt == "e2m1":
        amax = latent.abs().amax(dim=1, keepdim=True)
        e = torch.where(amax > 0, _power_of_two_below(amax, 10), torch.zeros_like(amax, dtype=torch.int32))
        x = torch.ldexp(latent, -e).view(n, 32, 16)
        s = (x.abs().amax(dim=2) / 6.0).to(torch.float8_e4m3fn)
        codes = _e2m1_codes(x, s.float()[:, :, None]).view(n, 256, 2)
        packed = (codes[:, :, 0] + 16 * codes[:, :, 1]).to(torch.uint8)
        row = torch.ldexp(torch.ones_like(amax), e).view(torch.uint8)
        return torch.cat([packed, s.view(torch.uint8), row, torch.zeros((n, 12), dtype=torch.uint8, device=DEV)], dim=1)
    if fmt == "e4m3":
        amax = latent.abs().amax(dim=1, keepdim=True)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        codes = (latent / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        return torch.cat([codes, scale.view(torch.uint8), torch.zeros((n, 12), dtype=torch.uint8, device=DEV)], dim=1)
    x = latent.view(n, 4, 128)
    amax = x.abs().amax(dim=2, keepdim=True)
    e = torch.where(amax > 0, _power_of_two_below(amax, 8), torch.full_like(amax, -127, dtype=torch.int32))
    codes = torch.ldexp(x, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).view(n, 512)
    return torch.cat([codes, torch.ldexp(torch.ones_like(amax), e).view(n, 4).view(torch.uint8)], dim=1)


def _write(latent, rope, fmt):
    """Cache rows (in the cache's storage type) of latent [n, 512] and rope [n, 64], both 32-bit values."""
    if fmt == "f32":
        return torch.cat([latent, rope], dim=1)
    if fmt == "bf16":
        return torch.cat([latent, rope], dim=1).to(torch.bfloat16)
    return torch.cat([_encode(latent, fmt), rope.to(torch.bfloat16).view(torch.uint8)], dim=1)


def _values(raw, fmt):
    """The 32-bit values [..., 576] that cache rows stand for."""
    if fmt in ("f32", "bf16"):
        return raw.float()
    rope = raw[..., -128:].contiguous().view(torch.bfloat16).float()
    if fmt == "e2m1":
        m = torch.tensor(E2M1_MAGNITUDES, device=DEV)
        table = torch.cat([m, -m])
        b = raw[..., :256].int()
        codes = table[torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)]
        s = raw[..., 256:288].contiguous().view(torch.float8_e4m3fn).float() * raw[..., 288:292].contiguous().view(torch.float32)
        return torch.cat([(codes.unflatten(-1, (32, 16)) * s[..., None]).flatten(-2), rope], dim=-1)
    codes = raw[..., :512].contiguous().view(torch.float8_e4m3fn).float()
    if fmt == "e4m3":
        return torch.cat([codes * raw[..., 512:516].contiguous().view(torch.float32), rope], dim=-1)
    s = raw[..., 512:528].contiguous().view(torch.float32)
    return torch.cat([(codes.unflatten(-1, (4, 128)) * s[..., None]).flatten(-2), rope], dim=-1)


def _rows(table, seq, pos):
    """Cache rows of positions pos [T, ...] of the sequences seq [T]."""
    page = table.long()[seq.long().view(-1, *([1] * (pos.dim() - 1))), (pos // PAGE).long()]
    return page * PAGE + (pos % PAGE).long()


# ------------------------------------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _latents(g, n):
    """Normalised latent vectors whose channels differ in size, as bf16 values."""
    gain = torch.exp(0.5 * torch.randn((1, D_LATENT), generator=g, device=DEV))
    return (torch.randn((n, D_LATENT), generator=g, device=DEV) * gain).to(torch.bfloat16)


def _pool(g, B, ctx):
    """A page table [B, pages] of shuffled pages, and the rows of the pool."""
    pages = (ctx + PAGE - 1) // PAGE
    table = torch.randperm(B * pages, generator=g, device=DEV).to(torch.int32).view(B, pages)
    return table, B * pages * PAGE


def _last_positions(B, per, ctx):
    """q_seq, q_pos of the last `per` tokens of every sequence."""
    seq = torch.arange(B, dtype=torch.int32, device=DEV).repeat_interleave(per)
    return seq, torch.arange(ctx - per, ctx, dtype=torch.int32, device=DEV).repeat(B)


_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rope_plan(dsa, d, scaling, layout):
    more = {"none": {}, "linear": dict(factor=32.0), "ntk": dict(factor=32.0),
            "yarn": dict(factor=32.0, original_ctx=4096)}[scaling]
    return dsa.Rope.make(d, theta=10000.0, layout=layout, scaling=scaling, device=DEV, **more)


def _handles(case, s):
    """The descriptors, rotation plan and scratch memory that a serving program keeps beside its tensors."""
    import dsa_indexed_sparse_gb300 as dsa
    if case["op"] == "rope":
        return dict(dsa=dsa, rope=_rope_plan(dsa, case["d"], case["scaling"], case["layout"]))
    seq = dsa.Seq(q_seq=s["seq"], q_pos=s["pos"], block_table=s["table"], max_ctx=case["ctx"],
                  cache_rows=s["cache"].shape[0], page_size=PAGE,
                  q_per_seq=case["T"] // case["B"] if case["op"] == "attention" else 0)
    code = {"bf16": None, "f32": None, "e4m3": dsa.DSA_E4M3, "e4m3_t128": dsa.DSA_E4M3_T128, "e2m1": dsa.DSA_E2M1}
    fmt = case.get("fmt", "e2m1")
    q = s.get("q")
    if q is None:   # the writers and the reader use the cache's layout only
        q = torch.empty((1, HEADS, D_ROW), dtype=torch.float32 if fmt == "f32" else torch.bfloat16, device=DEV)
    mla = dsa.Mla(q=q, kv_cache=s["cache"], d_latent=D_LATENT, d_rope=D_ROPE, softmax_scale=192 ** -0.5, dtype=code[fmt])
    h = dict(dsa=dsa, seq=seq, mla=mla)
    if case["op"] == "append":
        h["rope"] = _rope_plan(dsa, D_ROPE, case["scaling"], "interleaved")
    if case["op"] == "attention":
        n = dsa.sparse_mla_attn_workspace_size(seq, mla, case["K"])
        h["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return h


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "rope":
        T, H, d, dt = case["T"], case["H"], case["d"], _DTYPES[case["dtype"]]
        s["x"] = torch.randn((T, H, d), generator=g, device=DEV).to(dt)
        s["pos"] = torch.randint(0, case["ctx"], (T,), generator=g, device=DEV, dtype=torch.int32)
        row = max(case["out_row"], d)
        s["out"] = torch.zeros((T, H, row), dtype=dt, device=DEV)[..., row - d:]
    elif case["op"] == "append":
        fmt = case["fmt"]
        s["table"], rows = _pool(g, case["B"], case["ctx"])
        s["seq"], s["pos"] = _last_positions(case["B"], case["T"] // case["B"], case["ctx"])
        dt = torch.float32 if fmt == "f32" else torch.bfloat16
        s["latent"] = _latents(g, case["T"]).to(dt)
        # the rope part is a slice of the projection that made it, as the model computes it
        s["k_rope"] = torch.randn((case["T"], D_ROW), generator=g, device=DEV).to(dt)[:, D_LATENT:]
        if fmt in ("bf16", "f32"):
            s["cache"] = torch.randn((rows, D_ROW), generator=g, device=DEV).to(dt)
        else:
            s["cache"] = torch.zeros((rows, _row_bytes(fmt)), dtype=torch.uint8, device=DEV)
            s["out"] = torch.zeros((case["T"], D_ROW), dtype=torch.bfloat16, device=DEV)
    else:
        fmt = case.get("fmt", "e2m1")
        s["table"], rows = _pool(g, case["B"], case["ctx"])
        s["seq"], s["pos"] = _last_positions(case["B"], case["T"] // case["B"], case["ctx"])
        rope = torch.randn((rows, D_ROPE), generator=g, device=DEV).to(torch.bfloat16).float()
        s["cache"] = _write(_latents(g, rows).float(), rope, fmt)
        if case["op"] == "read":
            s["out"] = torch.zeros((case["T"], D_ROW), dtype=_DTYPES[case["dtype"]], device=DEV)
        else:
            T, K = case["T"], case["K"]
            s["q"] = torch.randn((T, HEADS, D_ROW), generator=g, device=DEV).to(torch.bfloat16)
            # a random choice of K of each query's causal positions, ascending, -1 behind them
            key = torch.rand((T, case["ctx"]), generator=g, device=DEV)
            key.masked_fill_(torch.arange(case["ctx"], device=DEV)[None, :] > s["pos"][:, None], 2.0)
            best, idx = key.topk(min(K, case["ctx"]), dim=1, largest=False)
            idx = torch.where(best < 2.0, idx, case["ctx"]).sort(dim=1).values
            idx = torch.nn.functional.pad(torch.where(idx < case["ctx"], idx, -1), (0, K - idx.shape[1]), value=-1)
            if case["holes"]:
                idx = torch.where(torch.rand((T, K), generator=g, device=DEV) < 0.2, -1, idx)
                idx[T // 2] = -1
            s["idx"] = idx.to(torch.int32).contiguous()
            s["out"] = torch.zeros((T, HEADS, D_LATENT), dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.zeros((T, HEADS), dtype=torch.float32, device=DEV)
    if own:
        s.update(_handles(case, s))
    return s


# ------------------------------------------------------------------------------------------------- one pass

def _run_own(s):
    c, dsa = s["case"], s["dsa"]
    if c["op"] == "rope":
        dsa.rope(s["rope"], s["pos"], s["x"], s["out"], inverse=c["inverse"])
        return s["out"]
    if c["op"] == "append":
        dsa.latent_cache_append_rope(s["seq"], s["mla"], s["rope"], s["latent"], s["k_rope"])
        if c["fmt"] in ("bf16", "f32"):
            return s["cache"]
        return dsa.latent_cache_read(s["seq"], s["mla"], s["out"])
    if c["op"] == "attention":
        dsa.sparse_mla_attn(s["seq"], s["mla"], s["idx"], c["K"], s["out"], lse=s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    return dsa.latent_cache_read(s["seq"], s["mla"], s["out"])


def _run_plain(s):
    c = s["case"]
    if c["op"] == "rope":
        f, m = _frequencies(c["d"], c["scaling"])
        s["out"].copy_(_rotate(s["x"].float(), s["pos"], f, m, c["layout"], c["inverse"]))
        return s["out"]
    row = _rows(s["table"], s["seq"], s["pos"])
    if c["op"] == "append":
        f, m = _frequencies(D_ROPE, c["scaling"])
        rope = _rotate(s["k_rope"].float(), s["pos"], f, m, "interleaved", False)
        s["cache"][row] = _write(s["latent"].float(), rope, c["fmt"])
        return s["cache"] if c["fmt"] in ("bf16", "f32") else _values(s["cache"][row], c["fmt"]).to(torch.bfloat16)
    if c["op"] == "read":
        return _values(s["cache"][row], c["fmt"]).to(s["out"].dtype)
    row = _rows(s["table"], s["seq"], s["idx"].clamp(min=0))
    if row.numel() > s["cache"].shape[0]:   # more selected rows than the pool holds: widen the pool once
        k = _values(s["cache"], "e2m1")[row]
    else:
        k = _values(s["cache"][row], "e2m1")
    logits = torch.matmul(s["q"].float(), k.transpose(1, 2)) * 192 ** -0.5
    logits = logits.masked_fill((s["idx"] < 0)[:, None, :], float("-inf"))
    top = logits.amax(dim=2, keepdim=True)
    p = (logits - torch.where(top > float("-inf"), top, torch.zeros_like(top))).exp()
    total = p.sum(dim=2, keepdim=True)
    out = torch.matmul(p, k[:, :, :D_LATENT]) / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": out.to(torch.bfloat16), "lse": (top + total.log())[:, :, 0]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------------- in 64 bits

def _rotate64(x, pos, freq, factor, layout, inverse):
    """The rotation as a product of complex numbers."""
    turn = torch.polar(torch.full_like(freq, factor)[None, :].expand(pos.shape[0], -1), pos.double()[:, None] * freq)
    turn = turn.conj() if inverse else turn
    x = x.double()
    pairs = x.unflatten(-1, (-1, 2)) if layout == "interleaved" else x.unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous()) * (turn[:, None, :] if x.dim() == 3 else turn)
    back = torch.view_as_real(z)
    return (back if layout == "interleaved" else back.transpose(-1, -2)).flatten(-2)


def _nearest64(x, top, mantissa, smallest):
    """x to the nearest number with `mantissa` bits behind the leading one, ties to even; below `smallest` (the least
    normal number) in its steps; magnitudes up to `top`."""
    step = torch.exp2(torch.frexp(x.abs().clamp(min=smallest))[1].double() - 1 - mantissa)
    return (torch.round(x / step) * step).clamp(-top, top)


def _stored64(latent, fmt):
    """The values that quantised latent rows hold."""
    x = latent.double()
    if fmt in ("f32", "bf16"):
        return x
    if fmt == "e4m3":
        scale = x.abs().amax(dim=1, keepdim=True) / 448.0
        scale = torch.where(scale > 0, scale, torch.ones_like(scale))
        scale = scale.float().double()   # stored in 32 bits; the format's quotient is formed in 32 bits too
        return _nearest64((x / scale).float().double(), 448.0, 3, 2.0 ** -6) * scale
    if fmt == "e4m3_t128":
        t = x.unflatten(1, (4, 128))
        scale = torch.exp2(torch.frexp(t.abs().amax(dim=2, keepdim=True).clamp(min=2.0 ** -119))[1].double() - 9)
        return (_nearest64(t / scale, 448.0, 3, 2.0 ** -6) * scale).flatten(1)
    row = torch.exp2(torch.frexp(x.abs().amax(dim=1, keepdim=True).clamp(min=2.0 ** -116))[1].double() - 11)
    t = (x / row).unflatten(1, (32, 16))
    scale = _nearest64(t.abs().amax(dim=2, keepdim=True) / 6.0, 448.0, 3, 2.0 ** -6)
    q = torch.where(scale > 0, t / torch.where(scale > 0, scale, torch.ones_like(scale)), torch.zeros_like(t))
    return (_nearest64(q, 6.0, 1, 1.0) * scale).flatten(1) * row


def _decoded64(raw, fmt):
    """The values [n, 576] that the bytes of cache rows stand for, from the formats' bit fields."""
    if fmt in ("f32", "bf16"):
        return raw.double()

    def small_float(code, exponent_bits, mantissa_bits, bias):
        code = code.long()
        e, m = (code >> mantissa_bits) & ((1 << exponent_bits) - 1), code & ((1 << mantissa_bits) - 1)
        one = float(1 << mantissa_bits)
        v = torch.where(e > 0, (1.0 + m.double() / one) * torch.exp2((e - bias).double()), m.double() / one * 2.0 ** (1 - bias))
        return torch.where((code >> (exponent_bits + mantissa_bits)) & 1 > 0, -v, v)
    rope = torch.stack([raw[:, -128::2].int(), raw[:, -127::2].int()], dim=2)
    rope = ((rope[:, :, 1] << 24) | (rope[:, :, 0] << 16)).view(torch.float32).double()
    if fmt == "e2m1":
        codes = torch.stack([raw[:, :256] & 15, raw[:, :256] >> 4], dim=2).flatten(1)
        scale = small_float(raw[:, 256:288], 4, 3, 7) * raw[:, 288:292].contiguous().view(torch.float32).double()
        v = small_float(codes, 2, 1, 1) * scale.repeat_interleave(16, dim=1)
    else:
        width = 128 if fmt == "e4m3_t128" else 512
        scale = raw[:, 512:512 + 2048 // width].contiguous().view(torch.float32).double()
        v = small_float(raw[:, :512], 4, 3, 7) * scale.repeat_interleave(width, dim=1)
    return torch.cat([v, rope], dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        f, m = _frequencies(case["d"], case["scaling"])
        return _rotate64(s["x"], s["pos"], f, m, case["layout"], case["inverse"])
    seq, pos, table = s["seq"].long(), s["pos"].long(), s["table"].long()
    row = table[seq, pos // PAGE] * PAGE + pos % PAGE
    if case["op"] == "append":
        f, m = _frequencies(D_ROPE, case["scaling"])
        new = torch.cat([_stored64(s["latent"], case["fmt"]),
                         _rotate64(s["k_rope"], s["pos"], f, m, "interleaved", False)], dim=1)
        if case["fmt"] in ("bf16", "f32"):
            pool = s["cache"].double()
            pool[row] = new
            return pool
        return new
    if case["op"] == "read":
        return _decoded64(s["cache"][row], case["fmt"])
    outs, lses = [], []
    step = max(1, (1 << 18) // case["K"])
    for a in range(0, case["T"], step):
        idx = s["idx"][a:a + step].long()
        at = idx.clamp(min=0)
        r = table[seq[a:a + step, None], at // PAGE] * PAGE + at % PAGE
        k = _decoded64(s["cache"][r.flatten()], "e2m1").view(*idx.shape, D_ROW)
        z = torch.einsum("thd,tkd->thk", s["q"][a:a + step].double(), k) / math.sqrt(192.0)
        z = torch.where(idx[:, None, :] >= 0, z, torch.full_like(z, float("-inf")))
        lse = torch.logsumexp(z, dim=2)
        p = torch.where(torch.isfinite(z), (z - torch.where(torch.isfinite(lse), lse, 0.0)[:, :, None]).exp(), 0.0)
        outs.append(torch.einsum("thk,tkd->thd", p, k[:, :, :D_LATENT]))
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
