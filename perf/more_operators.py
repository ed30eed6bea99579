"""The measured cases of the 4-bit index keys and of the attention over selected blocks: new keys quantised to MXFP4
into the paged cache and read back, index scores of queries quantised on the way, the choice of blocks (pages) by the
best score in each, and the attention over the chosen blocks.

Plain forms (``own`` false) are elementary torch operations in 32 bits; with ``own`` true ``run`` makes the calls a
user makes of ``dsa_indexed_sparse_gb300``.  The sizes are those of the decode and prefill configurations of this
repository: 64 indexer heads of 128, 128 attention heads over 512 latent + 64 rope dims, 64-token pages, 2048
selected rows (32 blocks).
"""
import math

import torch

own = False

D_LATENT, D_ROPE, HEADS, PAGE = 512, 64, 128, 64
D_ROW = D_LATENT + D_ROPE
H_I, D_I, GROUP = 64, 128, 32
SCALE = 192 ** -0.5
DEV = "cuda" if torch.cuda.is_available() else "cpu"
E2M1_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # the new tokens of a decode batch into the 4-bit key cache, read back as the values they stand for
        dict(name="keys decode 64", op="keys", T=64, B=64, ctx=8192, D=D_I, src="bf16", out="bf16"),
        # an odd chunk of seven sequences, fp32 keys as a normalisation in 32 bits leaves them
        dict(name="keys chunk 1001", op="keys", T=1001, B=7, ctx=4000, D=D_I, src="f32", out="f32"),
        # a whole prompt
        dict(name="keys prompt 16384", op="keys", T=16384, B=1, ctx=16384, D=D_I, src="bf16", out="bf16"),
        # one decode token over a 32768-token cache
        dict(name="scores decode 1", op="scores", T=1, B=1, ctx=32768),
        # long decode: four sequences of up to 131072 tokens
        dict(name="scores decode 4 long", op="scores", T=4, B=4, ctx=131072),
        # a prompt chunk at the end of 8192 tokens
        dict(name="scores chunk 2048", op="scores", T=2048, B=1, ctx=8192),
        # the blocks of one decode token: the smallest call
        dict(name="select decode 1", op="select", T=1, B=1, ctx=32768, blocks=32, first=1, last=2),
        # the blocks of a prompt chunk's queries
        dict(name="select chunk 4096", op="select", T=4096, B=1, ctx=16384, blocks=32, first=1, last=2),
        # one decode token over 32 of its 512 blocks
        dict(name="attention decode 1", op="attention", T=1, B=1, ctx=32768, blocks=32, holes=False),
        # a decode batch over caches of up to 8192 tokens
        dict(name="attention decode 64", op="attention", T=64, B=64, ctx=8192, blocks=32, holes=False),
        # an odd batch and an odd number of blocks, unused entries in the middle and a row that selects nothing
        dict(name="attention ragged 7x13", op="attention", T=7, B=7, ctx=3001, blocks=13, holes=True),
        # a causal prompt chunk: 2048 queries at the end of a 4096-token sequence
        dict(name="attention chunk 2048", op="attention", T=2048, B=1, ctx=4096, blocks=32, holes=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["keys", "scores", "select", "attention"])
    B = _spread(rng, 1, 64)
    if op == "keys":
        per = _spread(rng, 1, 16384 // B)
        return dict(op=op, T=B * per, B=B, ctx=per + _spread(rng, 1, 16384 // B), D=rng.choice([64, 128, 256]),
                    src=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
    if op == "scores":
        per = 1 if rng.random() < 0.5 else _spread(rng, 1, max(1, 2048 // B))
        return dict(op=op, T=B * per, B=B, ctx=per + _spread(rng, 16, min(131072, (13 << 20) // (B * per)) - per))
    if op == "select":
        per = 1 if rng.random() < 0.5 else _spread(rng, 1, max(1, 4096 // B))
        first, last = rng.choice([0, 1, 2]), rng.choice([0, 1, 2, 5])
        ctx = per + _spread(rng, 1024, min(262144, (48 << 20) // (B * per)) - per)
        free = min(120, ctx // PAGE * 3 // 4 - first - last)
        return dict(op=op, T=B * per, B=B, ctx=ctx, blocks=first + last + _spread(rng, 1, free), first=first, last=last)
    per = 1 if rng.random() < 0.5 else _spread(rng, 1, max(1, 2048 // B))
    blocks = _spread(rng, 1, min(256, 65536 // (B * per)))
    return dict(op=op, T=B * per, B=B, ctx=per + _spread(rng, 16, 131072 // B), blocks=blocks, holes=rng.random() < 0.4)


def _lengths(case):
    """Tokens that each sequence holds: the longest has ctx, the shortest about three quarters of it."""
    B, per, ctx = case["B"], case["T"] // case["B"], case["ctx"]
    return [max(per, ctx - (b * 37 % B) * ctx // (4 * B)) for b in range(B)]


def _pairs(case):
    """(query, causal position) pairs."""
    per = case["T"] // case["B"]
    return sum(n * per - per * (per - 1) // 2 for n in _lengths(case))


def work(case):
    T, op = case["T"], case["op"]
    if op == "keys":
        D = case["D"]
        size = {"bf16": 2, "f32": 4}
        return {"bytes": T * (D * size[case["src"]] + D // 2 + D // GROUP + D * size[case["out"]] + 8), "flops": 4 * T * D}
    if op == "scores":
        keys = sum(_lengths(case)) * (D_I // 2 + D_I // GROUP)
        return {"bytes": keys + T * H_I * (2 * D_I + 4) + 4 * _pairs(case), "flops": 2 * H_I * D_I * _pairs(case)}
    if op == "select":
        return {"bytes": 4 * _pairs(case) + 4 * T * case["blocks"], "flops": _pairs(case)}
    per = T // case["B"]
    rows = sum(min(PAGE * case["blocks"], n - per + i + 1) for n in _lengths(case) for i in range(per))
    distinct = min(rows, sum(_lengths(case)))
    return {"bytes": distinct * D_ROW * 2 + T * (HEADS * (D_ROW * 2 + D_LATENT * 2 + 4) + case["blocks"] * 4),
            "flops": 2 * HEADS * (D_ROW + D_LATENT) * rows}


# ------------------------------------------------------------------------------------------------- the format

def _power(e):
    """2^e in 32 bits, from its exponent bits (no less than 2^-126)."""
    return ((e.clamp(min=-126) + 127) << 23).view(torch.float32)


def _quantise(x):
    """MXFP4 of x [..., D] (32-bit values): bytes of two codes [..., D/2], exponent bytes [..., D/32]."""
    g = x.unflatten(-1, (-1, GROUP))
    amax = g.abs().amax(dim=-1, keepdim=True)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 1 - 2).clamp(-127, 127), -127)
    a = g.abs() * _power(-e.to(torch.int32))
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() +
            (a >= 3.5).int() + (a > 5.0).int() + 8 * torch.signbit(g).int()).flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), (e[..., 0] + 127).to(torch.uint8)


def _values(codes, exps):
    """The 32-bit values that bytes of two codes and their exponent bytes stand for."""
    m = torch.tensor(E2M1_MAGNITUDES, device=codes.device)
    b = codes.int()
    v = torch.cat([m, -m])[torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)]
    return (v.unflatten(-1, (-1, GROUP)) * _power(exps.int().unsqueeze(-1) - 127)).flatten(-2)


# ------------------------------------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _vectors(g, shape, D, dt):
    """Keys or query heads whose channels differ in size."""
    gain = torch.exp(0.5 * torch.randn((D,), generator=g, device=DEV))
    return (torch.randn((*shape, D), generator=g, device=DEV) * gain).to(dt)


def _pool(g, case):
    """A page table [B, pages] of shuffled pages, the rows of the pool, and the queries' sequences and positions: the
    last tokens of every sequence."""
    B, per, lens = case["B"], case["T"] // case["B"], _lengths(case)
    pages = (case["ctx"] + PAGE - 1) // PAGE
    table = torch.randperm(B * pages, generator=g, device=DEV).to(torch.int32).view(B, pages)
    end = torch.tensor(lens, dtype=torch.int32, device=DEV)
    seq = torch.arange(B, dtype=torch.int32, device=DEV).repeat_interleave(per)
    pos = (end[:, None] - per + torch.arange(per, dtype=torch.int32, device=DEV)[None, :]).flatten().contiguous()
    return table, B * pages * PAGE, seq, pos


def _handles(case, s):
    """The descriptors and scratch memory that a serving program keeps beside its tensors."""
    import dsa_indexed_sparse_gb300 as dsa
    per, op = case["T"] // case["B"], case["op"]
    seq = dsa.Seq(q_seq=s["seq"], q_pos=s["pos"], block_table=s["table"], max_ctx=case["ctx"], cache_rows=s["rows"],
                  page_size=PAGE, q_per_seq=per)
    h = dict(dsa=dsa, dsa_seq=seq)
    if op == "scores":
        h["codes"] = torch.empty((case["T"], H_I, D_I // 2), dtype=torch.uint8, device=DEV)
        h["exps"] = torch.empty((case["T"], H_I, D_I // GROUP), dtype=torch.uint8, device=DEV)
        h["index"] = dsa.Indexer(q=h["codes"], w=s["w"], k_cache=s["k_codes"], q_scale=h["exps"], k_scale=s["k_exps"],
                                 dtype=dsa.DSA_MXFP4_E2M1)
    if op == "attention":
        h["mla"] = dsa.Mla(q=s["q"], kv_cache=s["cache"], d_latent=D_LATENT, d_rope=D_ROPE, softmax_scale=SCALE)
        n = dsa.block_mla_attn_workspace_size(seq, h["mla"], case["blocks"])
        h["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return h


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    T, B, ctx, op = case["T"], case["B"], case["ctx"], case["op"]
    s["table"], s["rows"], s["seq"], s["pos"] = _pool(g, case)
    if op == "keys":
        s["new"] = _vectors(g, (T,), case["D"], _DTYPES[case["src"]])
        s["k_codes"] = torch.zeros((s["rows"], case["D"] // 2), dtype=torch.uint8, device=DEV)
        s["k_exps"] = torch.zeros((s["rows"], case["D"] // GROUP), dtype=torch.uint8, device=DEV)
        s["out"] = torch.zeros((T, case["D"]), dtype=_DTYPES[case["out"]], device=DEV)
    elif op == "scores":
        s["q"] = _vectors(g, (T, H_I), D_I, torch.bfloat16)
        s["w"] = torch.randn((T, H_I), generator=g, device=DEV) / 8.0
        s["k_codes"], s["k_exps"] = _quantise(_vectors(g, (s["rows"],), D_I, torch.float32))
        s["scores"] = torch.zeros((T, (ctx + 3) // 4 * 4), device=DEV)
    elif op == "select":
        # scores of nearby positions go together, as a text's do; some are equal; what lies behind a query's position
        # is left from earlier steps
        n = (ctx + 3) // 4 * 4
        common = torch.randn((T, (n + 15) // 16), generator=g, device=DEV).repeat_interleave(16, dim=1)[:, :n]
        s["scores"] = common.add_(torch.randn((T, n), generator=g, device=DEV)).to(torch.bfloat16).float().contiguous()
        s["scores"][torch.arange(n, device=DEV)[None, :] > s["pos"][:, None]] += 100.0
        s["chosen"] = torch.empty((T, case["blocks"]), dtype=torch.int32, device=DEV)
    else:
        s["cache"] = _vectors(g, (s["rows"],), D_ROW, torch.bfloat16)
        s["q"] = torch.randn((T, HEADS, D_ROW), generator=g, device=DEV).to(torch.bfloat16)
        # the query's own block and a random choice of the others that it may see, ascending, -1 behind them
        N, pages = case["blocks"], s["table"].shape[1]
        own_block = (s["pos"] // PAGE).long()
        key = torch.rand((T, pages), generator=g, device=DEV)
        key.scatter_(1, own_block[:, None], -1.0)
        key.masked_fill_(torch.arange(pages, device=DEV)[None, :] > own_block[:, None], 2.0)
        best, idx = key.topk(min(N, pages), dim=1, largest=False)
        idx = torch.where(best < 2.0, idx, pages).sort(dim=1).values
        idx = torch.nn.functional.pad(torch.where(idx < pages, idx, -1), (0, N - idx.shape[1]), value=-1)
        if case["holes"]:
            idx = torch.where(torch.rand((T, N), generator=g, device=DEV) < 0.2, -1, idx)
            idx[T // 2] = -1
        s["idx"] = idx.to(torch.int32).contiguous()
        s["out"] = torch.zeros((T, HEADS, D_LATENT), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros((T, HEADS), dtype=torch.float32, device=DEV)
    if own:
        s.update(_handles(case, s))
    return s


# ------------------------------------------------------------------------------------------------- one pass

def _run_own(s):
    c, dsa, seq = s["case"], s["dsa"], s["dsa_seq"]
    if c["op"] == "keys":
        dsa.index_cache_append(seq, s["new"], s["k_codes"], s["k_exps"], dtype=dsa.DSA_MXFP4_E2M1)
        return dsa.index_cache_read(seq, s["k_codes"], s["k_exps"], s["out"], dtype=dsa.DSA_MXFP4_E2M1)
    if c["op"] == "scores":
        dsa.index_query_quantize(s["q"], s["codes"], s["exps"], dtype=dsa.DSA_MXFP4_E2M1)
        return dsa.indexer_scores(seq, s["index"], s["scores"])
    if c["op"] == "select":
        return dsa.block_topk(seq, s["scores"], c["blocks"], s["chosen"], first=c["first"], last=c["last"])
    dsa.block_mla_attn(seq, s["mla"], s["idx"], s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _cache_rows(table, seq, pos):
    """Cache rows of positions pos [T, ...] of the sequences seq [T]."""
    page = table.long()[seq.long().view(-1, *([1] * (pos.dim() - 1))), (pos // PAGE).long()]
    return page * PAGE + (pos % PAGE).long()


def _plain_scores(s):
    c = s["case"]
    B, per, ctx = c["B"], c["T"] // c["B"], c["ctx"]
    q = _values(*_quantise(s["q"].float())).view(B, per, H_I, D_I)
    at = torch.arange(ctx, device=DEV).repeat(B, 1)
    row = _cache_rows(s["table"], torch.arange(B, device=DEV), at)
    k = _values(s["k_codes"][row], s["k_exps"][row]).transpose(1, 2)          # [B, D, ctx]
    out, pos = s["scores"].view(B, per, -1)[:, :, :ctx], s["pos"].view(B, per)
    step = max(1, (1 << 28) // (B * H_I * ctx))
    for a in range(0, per, step):
        n = min(step, per - a)
        d = torch.matmul(q[:, a:a + n].reshape(B, n * H_I, D_I), k).view(B, n, H_I, ctx).clamp_(min=0.0)
        i = torch.matmul(s["w"].view(B, per, 1, H_I)[:, a:a + n], d)[:, :, 0]
        part = out[:, a:a + n]
        part.copy_(torch.where(at[:, None, :] <= pos[:, a:a + n, None], i, part))
    return s["scores"]


def _plain_select(s):
    c = s["case"]
    T, N = c["T"], c["blocks"]
    x = s["scores"][:, :c["ctx"]]
    x = torch.where(torch.arange(c["ctx"], device=DEV)[None, :] <= s["pos"][:, None], x, float("-inf"))
    nb = s["table"].shape[1]
    best = torch.nn.functional.pad(x, (0, nb * PAGE - c["ctx"]), value=float("-inf")).view(T, nb, PAGE).amax(dim=2)
    block, mine = torch.arange(nb, device=DEV)[None, :], (s["pos"] // PAGE)[:, None]
    best = torch.where((block < c["first"]) | (block > mine - c["last"]), float("inf"), best)
    best = torch.where(block <= mine, best, float("-inf"))
    order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :N]
    order = torch.where(order <= mine, order, nb).sort(dim=1).values
    s["chosen"][:, order.shape[1]:] = -1
    s["chosen"][:, :order.shape[1]] = torch.where(order < nb, order, -1).to(torch.int32)
    return s["chosen"]


def _plain_attention(s):
    c = s["case"]
    step = max(1, (1 << 21) // (c["blocks"] * PAGE))
    inside = torch.arange(PAGE, device=DEV)
    for a in range(0, c["T"], step):
        idx = s["idx"][a:a + step]
        pos = (idx.clamp(min=0).unsqueeze(-1) * PAGE + inside).flatten(1)
        seen = (idx >= 0).repeat_interleave(PAGE, dim=1) & (pos <= s["pos"][a:a + step, None])
        k = s["cache"][_cache_rows(s["table"], s["seq"][a:a + step], torch.where(seen, pos, 0))].float()
        logits = torch.matmul(s["q"][a:a + step].float(), k.transpose(1, 2)) * SCALE
        logits = logits.masked_fill(~seen[:, None, :], float("-inf"))
        top = logits.amax(dim=2, keepdim=True)
        p = (logits - torch.where(top > float("-inf"), top, torch.zeros_like(top))).exp()
        total = p.sum(dim=2, keepdim=True)
        s["out"][a:a + step] = torch.matmul(p, k[:, :, :D_LATENT]) / torch.where(total > 0, total, torch.ones_like(total))
        s["lse"][a:a + step] = (top + total.log())[:, :, 0]
    return {"out": s["out"], "lse": s["lse"]}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "keys":
        row = _cache_rows(s["table"], s["seq"], s["pos"])
        s["k_codes"][row], s["k_exps"][row] = _quantise(s["new"].float())
        s["out"].copy_(_values(s["k_codes"][row], s["k_exps"][row]))
        return s["out"]
    return {"scores": _plain_scores, "select": _plain_select, "attention": _plain_attention}[op](s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------------- in 64 bits

def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _stored64(x):
    """The values nearest to x [..., D] in MXFP4: a power of two for 32 values, numbers of two significant bits down
    to steps of a half, at most 6."""
    g = x.double().unflatten(-1, (-1, GROUP))
    amax = g.abs().amax(dim=-1, keepdim=True)
    unit = _power64(torch.frexp(amax.clamp(min=2.0 ** -125))[1] - 3)
    y = g / unit
    step = torch.where(y.abs() < 2.0, 0.5, torch.where(y.abs() < 4.0, 1.0, 2.0))
    return ((torch.round(y / step) * step).clamp(-6.0, 6.0) * unit).flatten(-2)


def _decoded64(codes, exps):
    """The values that bytes of two codes (sign, two exponent bits of bias 1, one fraction bit) and exponents hold."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e > 0, (1.0 + 0.5 * m) * _power64(e - 1), 0.5 * m) * (1.0 - 2.0 * (c >> 3).double())
    return v * _power64(exps.long() - 127).repeat_interleave(GROUP, dim=-1)


def _exact_scores(case, s):
    out = s["scores"].double()
    per = case["T"] // case["B"]
    for b, n in enumerate(_lengths(case)):
        at = torch.arange(n, device=DEV)
        row = s["table"][b].long()[at // PAGE] * PAGE + at % PAGE
        k = _decoded64(s["k_codes"][row], s["k_exps"][row])
        step = max(1, (1 << 27) // (H_I * n))
        for a in range(b * per, (b + 1) * per, step):
            z = min(a + step, (b + 1) * per)
            d = torch.einsum("thd,nd->thn", _stored64(s["q"][a:z]), k)
            i = torch.einsum("th,thn->tn", s["w"][a:z].double(), torch.relu(d))
            seen = at[None, :] <= s["pos"][a:z, None]
            out[a:z, :n] = torch.where(seen, i, out[a:z, :n])
    return out


def _exact_select(case, s):
    T, N = case["T"], case["blocks"]
    out = torch.full((T, N), -1, dtype=torch.int32, device=DEV)
    x = s["scores"].double()
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % PAGE)).unflatten(1, (-1, PAGE))
    at = torch.arange(x.shape[1] * PAGE, device=DEV).view(1, -1, PAGE)
    best = torch.where(at <= s["pos"][:, None, None], x, float("-inf")).amax(dim=2)
    nb = best.shape[1]
    block = torch.arange(nb, device=DEV)
    step = max(1, (1 << 27) // (nb * nb))
    for a in range(0, T, step):
        mine = (s["pos"][a:a + step] // PAGE)[:, None]
        v = best[a:a + step]
        there = block[None, :] <= mine
        forced = there & ((block[None, :] < case["first"]) | (block[None, :] > mine - case["last"]))
        v = torch.where(forced, float("inf"), v)
        # how many come before a block: those of a higher score, and of the same score those of a lower number
        before = (v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & (block[None, None, :] < block[None, :, None]))
        taken = there & ((before & there[:, None, :]).sum(dim=2) < N)
        place = taken.long().cumsum(dim=1) - 1
        t, j = taken.nonzero(as_tuple=True)
        out[a + t, place[t, j]] = j.to(torch.int32)
    return out


def _exact_attention(case, s):
    outs, lses = [], []
    N = case["blocks"]
    step = max(1, (1 << 18) // (N * PAGE))
    table, inside = s["table"].long(), torch.arange(PAGE, device=DEV)
    for a in range(0, case["T"], step):
        idx, seq, last = s["idx"][a:a + step].long(), s["seq"][a:a + step].long(), s["pos"][a:a + step]
        page = table[seq[:, None], idx.clamp(min=0)]
        k = s["cache"].view(-1, PAGE, D_ROW)[page].flatten(1, 2).double()                 # [t, N * 64, 576]
        seen = ((idx >= 0)[:, :, None] & (idx[:, :, None] * PAGE + inside <= last[:, None, None])).flatten(1)
        z = torch.einsum("thd,tkd->thk", s["q"][a:a + step].double(), k) / math.sqrt(192.0)
        z = torch.where(seen[:, None, :], z, float("-inf"))
        lse = torch.logsumexp(z, dim=2)
        p = torch.where(seen[:, None, :], (z - torch.where(torch.isfinite(lse), lse, 0.0)[:, :, None]).exp(), 0.0)
        outs.append(torch.einsum("thk,tkd->thd", p, k[:, :, :D_LATENT]))
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "keys":
        return _stored64(s["new"])
    return {"scores": _exact_scores, "select": _exact_select, "attention": _exact_attention}[case["op"]](case, s)
