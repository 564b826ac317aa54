"""The operators of serving a DART layer from a paged memory cache: what each computes, and the calls that measure it.

  write / round trip  finished chunk memories go into the pages of their sequences, as they are or as 4-bit codes with
                      a power-of-two scale for every 32 values, and come back out;
  read                the memories of a set of sequences gathered from their pages (and widened);
  extend              a run of new tokens per sequence through the recurrence, from the middle of a chunk on: outputs,
                      the new state, and the memories that close on the way, appended to the pages;
  sma                 state-memory attention of those tokens over the paged memories.

`run` computes them in elementary torch operations in float32 (decays in float64), or with `own` set through
mamba_ssd_state_b200.dart.  Tokens of all sequences are packed along one axis, sequence b owning rows
cu_tokens[b] .. cu_tokens[b+1]-1.  Memory m of sequence b is slot m % R of page table[b, m // R].

4-bit format of one memory V[N, P]: the 32 values V[32 k .. 32 k + 31, p] share the scale 2^(s - 127), s the byte
scales[p, k]; the codes are E2M1 (sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, low nibble first, the code of
V[16 i + 4 q + j, p] at place q (N / 4) + 4 i + j of row p.
"""
import math
import random

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GATE = 0.5


# ---------------------------------------------------------------- the cases
def listed():
    big = dict(heads=32, groups=1, dstate=128, headdim=64)
    return [
        # one sequence, one token, one finished memory and another half way: the first steps of a chat, all latency
        dict(name="sma one token", op="sma", seqs=1, tokens=1, mems=4, page=4, cache="bf16", dtype="bf16", **big),
        # the decode workload: 64 sequences of one token against 128 memories (32k tokens of context) each
        dict(name="sma decode batch", op="sma", seqs=64, tokens=1, mems=128, page=16, cache="bf16", dtype="bf16", **big),
        # drafted tokens of 32 sequences of different lengths, checked in one pass over 4-bit memories
        dict(name="sma drafts, 4-bit", op="sma", seqs=32, tokens=6, mems=131, page=16, cache="mxfp4", dtype="bf16", **big),
        # the next piece of four long prompts: hundreds of new tokens against up to 100 memories
        dict(name="sma prompt pieces", op="sma", seqs=4, tokens=256, mems=100, page=8, cache="bf16", dtype="bf16", **big),
        # float32 layers with grouped C and pages of an odd number of memories
        dict(name="sma float32, groups", op="sma", seqs=7, tokens=5, mems=45, page=7, cache="f32", dtype="f32",
             heads=8, groups=4, dstate=64, headdim=64),
        # the recurrence of a decode batch: one token a sequence
        dict(name="extend decode batch", op="extend", seqs=64, tokens=1, mems=6, page=4, cache="bf16", dtype="bf16", chunk=256, **big),
        # five drafted tokens of one sequence, over a chunk boundary
        dict(name="extend five drafts", op="extend", seqs=1, tokens=5, mems=3, page=2, cache="f32", dtype="f32", chunk=64,
             heads=8, groups=2, dstate=64, headdim=64),
        # the next piece of four prompts, each closing a chunk or more on the way
        dict(name="extend prompt pieces", op="extend", seqs=4, tokens=256, mems=8, page=8, cache="bf16", dtype="bf16", chunk=128, **big),
        # memories of two prompts of up to 31 chunks, kept as 4-bit codes, and read back
        dict(name="4-bit round trip", op="trip", seqs=2, mems=31, page=16, cache="mxfp4", dtype="bf16", **big),
        # one finished memory of every sequence of a batch into its page
        dict(name="write one memory", op="write", seqs=24, mems=1, page=4, cache="bf16", dtype="bf16", **big),
        # sequences that leave a 4-bit cache: their memories as dense bfloat16
        dict(name="read 4-bit", op="read", seqs=16, mems=63, page=16, cache="mxfp4", dtype="bf16", **big),
        # a few float32 memories of a small layer
        dict(name="read float32", op="read", seqs=3, mems=5, page=3, cache="f32", dtype="f32",
             heads=4, groups=1, dstate=16, headdim=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sma", "sma", "sma", "extend", "extend", "trip", "write", "read"])
    dstate, headdim = rng.choice([(128, 64), (128, 64), (64, 64), (16, 16)])
    cache = rng.choice(["bf16", "f32"] if dstate == 16 else ["bf16", "bf16", "mxfp4", "f32"])
    if op == "trip":
        cache, (dstate, headdim) = "mxfp4", rng.choice([(128, 64), (64, 64)])
    if op in ("extend", "write") and cache == "mxfp4":
        cache = "bf16"
    heads = rng.choice([2, 4, 8, 16, 32])
    case = dict(op=op, seqs=_log(rng, 1, 64), mems=_log(rng, 1, 160), page=rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 17]), cache=cache,
                dtype=rng.choice(["bf16", "f32"]) if cache == "mxfp4" else cache, heads=heads,
                groups=rng.choice([g for g in (1, 2, 4, 8) if heads % g == 0]), dstate=dstate, headdim=headdim)
    if op in ("sma", "extend"):
        case["tokens"] = _log(rng, 1, 256)
    if op == "extend":
        case["chunk"] = rng.choice([4, 32, 64, 100, 128, 256])
        case["mems"] = min(case["mems"], 20)
    # no more memories than the decode batch reads, no more products than the prompt pieces make
    while (case["seqs"] * case["mems"] * heads * dstate * headdim > 5e8
           or case["seqs"] * case.get("tokens", 1) * case["mems"] * heads * headdim * dstate > 2e10
           or case["seqs"] * case.get("tokens", 1) ** 2 * heads > 4e6 and op == "extend"):
        case["seqs"] = max(1, case["seqs"] // 2)
        case["mems"] = max(1, case["mems"] * 3 // 4)
    return case


def _lengths(n, most):
    """n lengths up to `most`, one of them `most` and, of five or more that are not all ones, one 0: batches are ragged."""
    if n == 1 or most == 1:
        return [most] * n
    got = [max(1, most - (b * 37) % (most // 2 + 1)) for b in range(n)]
    if n >= 5:
        got[3] = 0
    return got


def _plan(case):
    """What a case's sequences hold, from its numbers alone: tokens, memories and places in the chunk."""
    B = case["seqs"]
    toks = _lengths(B, case.get("tokens", 1))
    if case["op"] == "extend":
        S = case["chunk"]
        pos = [(S - 1 - 3 * b) % S if b % 2 else (S - 2 - b) % S for b in range(B)]
        n = [m - (b % 2) for b, m in enumerate(_lengths(B, case["mems"]))]
        n = [max(0, v) for v in n]
        closes = [(pos[b] + toks[b]) // S for b in range(B)]
        return toks, n, pos, closes
    return toks, _lengths(B, case["mems"])[::-1], [0] * B, [0] * B


# ------------------------------------------------------------------ inputs
def _type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def index(values):
        return torch.tensor(values, dtype=torch.int64, device="cuda")

    B, H, G, N, P, R = (case[k] for k in ("seqs", "heads", "groups", "dstate", "headdim", "page"))
    T = _type(case["dtype"])
    toks, n, pos, closes = _plan(case)
    need = [-(-(n[b] + closes[b]) // R) for b in range(B)]
    width = max(1, max(need))
    npages = sum(need) + 3
    order = torch.randperm(npages, generator=g, device="cuda").to(torch.int32)
    at = [sum(need[:b]) for b in range(B)]
    rows = index([[min(at[b] + k, npages - 1) for k in range(width)] for b in range(B)])
    there = index([[int(k < need[b]) for k in range(width)] for b in range(B)])
    s = dict(case=case, table=torch.where(there > 0, order[rows], -1).contiguous(), scales=None, n=ints(n))
    # the pool: memories of sums over a chunk, as large as the decode workload's
    if case["cache"] == "mxfp4":
        s["pages"] = torch.empty((npages, H, R, P, N // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((npages, H, R, P, N // 32), dtype=torch.uint8, device="cuda")
        some = max(1, (1 << 26) // (H * R * N * P))
        for k in range(0, npages, some):
            m = min(some, npages - k)
            s["pages"][k:k + m], s["scales"][k:k + m] = _encode(normal(m, H, R, N, P, scale=N ** -0.5))
    else:
        s["pages"] = torch.empty((npages, H, R, N, P), dtype=_type(case["cache"]), device="cuda")
        some = max(1, (1 << 28) // (H * R * N * P))
        for k in range(0, npages, some):
            s["pages"][k:k + some] = normal(min(some, npages - k), H, R, N, P, scale=N ** -0.5)
    if case["op"] in ("trip", "write", "read"):
        C = case["mems"]
        s["first"], s["count"] = ints([0] * B), ints(n)
        if case["op"] != "read":
            s["dH"] = normal(B, H, C, N, P, scale=N ** -0.5, dtype=T)
        if case["op"] != "write":
            s["out"] = torch.zeros((B, H, C, N, P), dtype=T, device="cuda")
        each = [(b, i) for b in range(B) for i in range(n[b])]
        s["each_b"], s["each_i"] = index([b for b, i in each]), index([i for b, i in each])
        return s
    rows = sum(toks)
    starts = [sum(toks[:b]) for b in range(B + 1)]
    s["cu"] = ints(starts)
    s["most"] = max(toks)
    s["own_row"] = index([b * s["most"] + i for b in range(B) for i in range(toks[b])])
    s["row"] = index([[min(starts[b] + i, max(rows - 1, 0)) for i in range(s["most"])] for b in range(B)])
    s["real"] = torch.tensor([[i < toks[b] for i in range(s["most"])] for b in range(B)], device="cuda")
    s["Cm"] = normal(rows, G, N, scale=N ** -0.5, dtype=T)
    if case["op"] == "sma":
        s["Q"] = normal(rows, H, N, scale=3.0, dtype=T)
        s["E"] = normal(rows, H, P, scale=P ** -0.5, dtype=T)
        s["y"] = normal(rows, H, P, scale=1 / 16)   # about what the attention adds
        # a chunk ends inside most runs of several tokens: their first half sees one memory less
        s["seen"] = ints([max(0, n[b] - (2 * i < toks[b] and toks[b] > 1)) for b in range(B) for i in range(toks[b])])
        return s
    s["x"] = normal(rows, H, P, dtype=T)
    s["Bm"] = normal(rows, G, N, scale=N ** -0.5, dtype=T)
    span = math.log(1e-1) - math.log(1e-3)
    s["dt"] = torch.exp(torch.rand((rows, H), generator=g, device="cuda") * span + math.log(1e-3))
    s["A"] = -torch.exp(torch.rand((H,), generator=g, device="cuda") * math.log(16.0))
    s["state"], s["cur"] = normal(B, H, N, P, scale=N ** -0.5), normal(B, H, N, P, scale=N ** -0.5)
    s["state_out"], s["cur_out"] = torch.empty_like(s["state"]), torch.empty_like(s["cur"])
    s["pos"], s["tokens"], s["closed"] = ints(pos), ints(toks), ints(closes)
    each = [(b, i) for b in range(B) for i in range(closes[b])]
    s["each_b"], s["each_i"], s["parts"] = index([b for b, i in each]), index([i for b, i in each]), max(closes) + 1
    return s


# ---------------------------------------------- the operators in plain form
def _power(k):
    """2^k in float32, exactly, for whole k from -126 to 127."""
    return ((k.int() + 127) << 23).view(torch.float32)


def _encode(V):
    """Codes and scales of memories V[..., N, P] in float32."""
    N, P = V.shape[-2:]
    blocks = V.reshape(*V.shape[:-2], N // 32, 32, P)
    most = blocks.abs().amax(-2)                                                    # [..., N/32, P]
    f, e = torch.frexp(most)
    k = torch.where(f <= 0.75, e - 3, e - 2).clamp(-126, 126)                       # the least k with most <= 6 * 2^k
    k = torch.where(most == 0, -126, k)
    fine = torch.isfinite(blocks).all(-2)
    a = blocks.abs() * _power(-k).unsqueeze(-2)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))                # between neighbours at a
    near = torch.round(a / step) * step                                             # a tie goes to the even code
    mark = torch.where(near < 2.0, 2.0 * near, torch.where(near < 4.0, near + 2.0, 0.5 * near + 4.0))
    mark = torch.where(fine.unsqueeze(-2), mark, 0.0).to(torch.uint8) + 8 * torch.signbit(blocks).to(torch.uint8)
    mark = torch.where(fine.unsqueeze(-2), mark, 0)
    scale = torch.where(fine, k + 127, 255).to(torch.uint8)
    mark = mark.reshape(*V.shape[:-2], N // 16, 4, 4, P).movedim(-1, -4).transpose(-3, -2)   # [..., P, q, i, j]
    mark = mark.reshape(*V.shape[:-2], P, N // 2, 2)
    return mark[..., 0] + 16 * mark[..., 1], scale.movedim(-1, -2).contiguous()


def _decode(codes, scales):
    """Memories [..., N, P] in float32 that codes [..., P, N/2] and scales [..., P, N/32] stand for."""
    P, half = codes.shape[-2:]
    N = 2 * half
    both = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 4, N // 16, 4)
    both = both.transpose(-3, -2).reshape(*codes.shape[:-1], N // 32, 32)           # by n
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    scale = torch.where(scales == 255, float("nan"), _power(scales.int() - 127))
    value = level[both.int()] * scale.unsqueeze(-1)
    return value.reshape(*codes.shape[:-1], N).transpose(-1, -2)


def _memories(s):
    """Every sequence's memories [B, H, M, N, P] in float32, M the slots of its table."""
    at = s["table"].clamp_min(0).long()
    got = s["pages"][at] if s["scales"] is None else _decode(s["pages"][at], s["scales"][at])
    B, W, H, R, N, P = got.shape
    return got.float().transpose(1, 2).reshape(B, H, W * R, N, P)


def _heads(v, H):
    """[..., G, N] with every group repeated for its heads."""
    return v.float().repeat_interleave(H // v.shape[-2], -2)


def _plain_sma(s):
    H, N = s["case"]["heads"], s["case"]["dstate"]
    mem = _memories(s)
    held = torch.arange(mem.shape[2], device="cuda") < s["n"][:, None]               # [B, M]
    mem = torch.where(held[:, None, :, None, None], mem, 0.0)
    Q, E, C = s["Q"].float()[s["row"]], s["E"].float()[s["row"]], _heads(s["Cm"], H)[s["row"]]
    U = torch.einsum("bthn,bhmnp->bthmp", Q, mem)
    score = torch.einsum("bthmp,bthp->bthm", U, E) / math.sqrt(N)
    del U
    seen = torch.arange(mem.shape[2], device="cuda") < s["seen"][s["row"]][..., None]   # [B, t, M]
    score = torch.where(seen[:, :, None], score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total > 0, total, 1.0)
    V = torch.einsum("bthn,bhmnp->bthmp", C, mem)
    o = torch.einsum("bthm,bthmp->bthp", w, V)
    return s["y"] + GATE * o.flatten(0, 1)[s["own_row"]]


def _plain_extend(s):
    case = s["case"]
    H, S, R, J = case["heads"], case["chunk"], case["page"], s["parts"]
    row, real, m = s["row"], s["real"], s["most"]
    x, Bh, Ch = s["x"].float()[row], _heads(s["Bm"], H)[row], _heads(s["Cm"], H)[row]
    dt = torch.where(real[..., None], s["dt"][row], 0.0)
    cum = torch.cumsum(dt.double() * s["A"].double(), 1)                             # [B, t, H]
    step = torch.arange(m, device="cuda")
    part = torch.div(s["pos"][:, None] + step, S, rounding_mode="floor")             # the chunk a token is in
    decay = torch.exp((cum[:, :, None] - cum[:, None]).clamp_max(0.0)).float() * dt[:, None]
    decay = torch.where((step[:, None] >= step)[None, :, :, None], decay, 0.0)
    gram = torch.einsum("bthn,bshn->btsh", Ch, Bh)
    y = torch.einsum("btsh,bshp->bthp", gram * decay, x)
    y = y + torch.exp(cum).float()[..., None] * torch.einsum("bthn,bhnp->bthp", Ch, s["state"])
    last = cum[:, -1]                                                                # padding adds nothing
    weight = torch.exp(last[:, None] - cum).float() * dt
    state = torch.exp(last).float()[..., None, None] * s["state"] + torch.einsum("bshn,bshp->bhnp", Bh, weight[..., None] * x)
    # every part of a chunk that the run passes: its memory at the chunk's last token, or at the run's
    place = torch.arange(J, device="cuda")
    ends = torch.minimum((place + 1) * S - 1 - s["pos"][:, None], s["tokens"][:, None] - 1).clamp_min(0).long()
    end = torch.gather(cum, 1, ends[..., None].expand(-1, -1, H))                    # [B, J, H]
    inside = (part[:, None] == place[:, None]) & real[:, None]                       # [B, J, s]
    weight = torch.exp((end[:, :, None] - cum[:, None]).clamp_max(0.0)).float() * dt[:, None]
    weight = torch.where(inside[..., None], weight, 0.0)
    D = torch.einsum("bjsh,bshn,bshp->bjhnp", weight, Bh, x)
    ran = (s["tokens"] > 0)[:, None, None, None]
    D[:, 0] += torch.where(ran, torch.exp(end[:, 0]).float()[..., None, None], 1.0) * s["cur"]
    slot = s["n"].long()[s["each_b"]] + s["each_i"]
    page = s["table"].long()[s["each_b"], torch.div(slot, R, rounding_mode="floor")]
    s["pages"][page, :, slot % R] = D[s["each_b"], s["each_i"]].to(s["pages"].dtype)
    cur = torch.gather(D, 1, s["closed"].long()[:, None, None, None, None].expand(-1, 1, *D.shape[2:]))[:, 0]
    seen = (s["n"][:, None] + part).flatten()[s["own_row"]].to(torch.int32)
    total = s["pos"] + s["tokens"]
    return dict(y=y.flatten(0, 1)[s["own_row"]], state=state, dH_cur=cur, nchunks=s["n"] + s["closed"],
                pos=total - s["closed"] * S, mem_count=seen, pages=s["pages"])


def _plain_write(s):
    slot = s["first"].long()[s["each_b"]] + s["each_i"]
    R = s["case"]["page"]
    page = s["table"].long()[s["each_b"], torch.div(slot, R, rounding_mode="floor")]
    if s["scales"] is None:
        s["pages"][page, :, slot % R] = s["dH"][s["each_b"], :, s["each_i"]].to(s["pages"].dtype)
        return
    codes, scales = _encode(s["dH"].float())
    s["pages"][page, :, slot % R] = codes[s["each_b"], :, s["each_i"]]
    s["scales"][page, :, slot % R] = scales[s["each_b"], :, s["each_i"]]


def _plain_read(s):
    slot = s["first"].long()[s["each_b"]] + s["each_i"]
    R = s["case"]["page"]
    page = s["table"].long()[s["each_b"], torch.div(slot, R, rounding_mode="floor")]
    got = s["pages"][page, :, slot % R]
    if s["scales"] is not None:
        got = _decode(got, s["scales"][page, :, slot % R])
    s["out"][s["each_b"], :, s["each_i"]] = got.to(s["out"].dtype)
    return s["out"]


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "sma":
            return _plain_sma(s)
        if case["op"] == "extend":
            return _plain_extend(s)
        if case["op"] != "read":
            _plain_write(s)
        return s["pages"] if case["op"] == "write" else _plain_read(s)
    from mamba_ssd_state_b200 import dart
    if case["op"] == "sma":
        return dart.dart_sma_paged(s["Q"], s["E"], s["Cm"], s["cu"], s["pages"], s["table"], s["seen"], GATE, s["y"], scales=s["scales"])
    if case["op"] == "extend":
        got = dart.dart_ssd_extend(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["cu"], s["state"], s["cur"], s["pages"], s["table"],
                                   s["n"], s["pos"], case["chunk"], scales=s["scales"], state_out=s["state_out"], dH_cur_out=s["cur_out"])
        return dict(got, pages=s["pages"])
    if case["op"] != "read":
        dart.dart_cache_write_paged(s["dH"], s["first"], s["count"], s["pages"], s["table"], scales=s["scales"])
        if case["op"] == "write":
            return s["pages"]
    return dart.dart_cache_read_paged(s["pages"], s["table"], s["first"], s["count"], scales=s["scales"], out=s["out"])


# ------------------------------------------------------- bytes and products
def work(case):
    B, H, G, N, P = (case[k] for k in ("seqs", "heads", "groups", "dstate", "headdim"))
    toks, n, pos, closes = _plan(case)
    T = 2 if case["dtype"] == "bf16" else 4
    one = {"bf16": 2 * N * P, "f32": 4 * N * P, "mxfp4": N * P // 2 + N * P // 32}[case["cache"]]
    if case["op"] in ("trip", "write", "read"):
        dense = T * N * P
        moved = {"trip": 2 * dense + one, "write": dense + one, "read": dense + one}[case["op"]]
        return {"bytes": sum(n) * H * moved, "flops": 0}
    rows = sum(toks)
    if case["op"] == "sma":
        held = [v if t else 0 for v, t in zip(n, toks)]
        less = [2 * max(0, n[b] - 1) * ((t + 1) // 2) + 2 * n[b] * (t // 2) if t > 1 else 2 * t * n[b] for b, t in enumerate(toks)]
        return {"bytes": sum(held) * H * one + rows * (H * (N + P) * T + G * N * T + 8 * H * P + 4),
                "flops": 2 * N * P * H * sum(less)}
    return {"bytes": 16 * B * H * N * P + rows * (H * P * T + 2 * G * N * T + 4 * H + 4 * H * P + 4) + sum(closes) * H * one,
            "flops": 4 * N * P * H * rows}


# ------------------------------------ the definitions, one by one, in 64 bits
def _power64(k):
    """2^k in float64, exactly, for whole k from -1022 to 1023."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _value64(s):
    """[pages, H, R, N, P] -> a function that gives memory `slot` of sequence b as [H, N, P] in float64."""
    R = s["case"]["page"]
    table = s["table"].tolist()
    sign_level = [(-1.0 if c >= 8 else 1.0) * LEVELS[c % 8] for c in range(16)]
    level = torch.tensor(sign_level, dtype=torch.float64, device="cuda")

    def of(b, slots):
        out = []
        for m in slots:
            page = s["pages"][table[b][m // R], :, m % R]
            if s["scales"] is None:
                out.append(page.double())
                continue
            H, P, half = page.shape
            N = 2 * half
            codes = torch.empty((H, P, N), dtype=torch.int64, device="cuda")
            codes[..., 0::2], codes[..., 1::2] = (page & 15).long(), (page >> 4).long()
            n = torch.arange(N, device="cuda")
            place = (n % 16 // 4) * (N // 4) + 4 * (n // 16) + n % 4
            power = _power64(s["scales"][table[b][m // R], :, m % R].long() - 127)
            out.append((level[codes[..., place]] * power[..., n // 32]).transpose(1, 2))
        return torch.stack(out, 1)

    return of


def _nearest64(V):
    """Each of V[..., N, P] in float64 as the nearest value its block's scale allows."""
    N, P = V.shape[-2:]
    block = V.reshape(*V.shape[:-2], N // 32, 32, P)
    most = block.abs().amax(-2, keepdim=True)
    k = torch.ceil(torch.log2(most / 6.0)).clamp(-126, 126).long()
    k = torch.where(6.0 * _power64(k - 1) >= most, k - 1, torch.where(6.0 * _power64(k) < most, k + 1, k)).clamp(-126, 126)
    unit = _power64(k)
    level = torch.tensor(LEVELS, dtype=torch.float64, device=V.device)
    off = (block.abs().unsqueeze(-1) - level * unit.unsqueeze(-1)).abs()
    odd = torch.arange(8, device=V.device) % 2
    best = torch.where(off == off.amin(-1, keepdim=True), odd, 9).argmin(-1)        # of two as near, the even code
    near = level[best]
    return torch.where(most > 0, torch.copysign(near, block) * unit, 0.0).reshape(V.shape)


def exact(case, seed):
    s = prepare(case, seed)
    H, N, G = case["heads"], case["dstate"], case["groups"]
    toks, n, pos, closes = _plan(case)
    B, R = case["seqs"], case["page"]
    of = _value64(s)
    table = s["table"].tolist()
    if case["op"] == "write":
        out = s["pages"].double()
        for b in range(B):
            for i in range(n[b]):
                out[table[b][i // R], :, i % R] = s["dH"][b, :, i].double()
        return out
    if case["op"] in ("trip", "read"):
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for b in range(B):
            if n[b]:
                out[b, :, :n[b]] = of(b, range(n[b])) if case["op"] == "read" else _nearest64(s["dH"][b, :, :n[b]].double())
        return out
    group = [h // (H // G) for h in range(H)]
    cu = [sum(toks[:b]) for b in range(B + 1)]
    if case["op"] == "sma":
        out = s["y"].double()
        seen = s["seen"].tolist()
        for b in range(B):
            if not toks[b] or not n[b]:
                continue
            mem = of(b, range(n[b]))                                                 # [H, M, N, P]
            for t in range(cu[b], cu[b + 1], 64):
                e = min(t + 64, cu[b + 1])
                key = torch.einsum("hmnp,thp->thmn", mem, s["E"][t:e].double())
                score = (key * s["Q"][t:e].double()[:, :, None]).sum(-1) / math.sqrt(N)
                hide = torch.arange(n[b], device="cuda") >= torch.tensor(seen[t:e], device="cuda")[:, None]
                score = score.masked_fill(hide[:, None], float("-inf"))
                w = torch.softmax(score, -1)
                w = torch.where(torch.isnan(w), 0.0, w)                              # nothing seen: nothing read
                mix = torch.einsum("thm,hmnp->thnp", w, mem)
                out[t:e] += GATE * torch.einsum("thn,thnp->thp", s["Cm"][t:e].double()[:, group], mix)
        return out
    # extend: token by token
    S = case["chunk"]
    state, cur = s["state"].double(), s["cur"].double()
    y = torch.zeros((sum(toks), H, case["headdim"]), dtype=torch.float64, device="cuda")
    pages = s["pages"].double()
    x, Bm, Cm = s["x"].double(), s["Bm"].double()[:, group], s["Cm"].double()[:, group]
    dt, A = s["dt"].double(), s["A"].double()
    n, pos = list(n), list(pos)
    for i in range(max(toks)):
        b = [k for k in range(B) if toks[k] > i]
        t = [cu[k] + i for k in b]
        a = torch.exp(dt[t] * A)[..., None, None]
        new = dt[t][..., None, None] * Bm[t][..., None] * x[t][:, :, None]
        state[b] = a * state[b] + new
        cur[b] = a * cur[b] + new
        y[t] = (state[b] * Cm[t][..., None]).sum(2)
        for k in b:
            pos[k] += 1
            if pos[k] == S:
                pages[table[k][n[k] // R], :, n[k] % R] = cur[k]
                cur[k] = 0.0
                n[k], pos[k] = n[k] + 1, 0
    return dict(y=y, state=state, dH_cur=cur, nchunks=None, pos=None, mem_count=None, pages=pages)


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(k)) for k in range(3)]:
        print(c, work(c))
