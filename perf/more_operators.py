"""What a step from token to token takes beside the ternary linears, the norm,
the cache's append and attention, and sampling: four operators as measured cases.

The lookup in the int8 embedding table, the per-head norm and rotary positions
of queries and keys, a ternary linear with bias, activation, gate and residual
in its epilogue, and the pages under the cache (forked, reserved, freed,
compacted and copied).  Geometries are the 8B's (hidden 4,096, FFN 12,288, 32
query and 8 key/value heads of 128, vocabulary 151,936, 36 layers), with
generic ones beside them.
"""
import math
import random

import torch

own = False
DEV = "cuda:0"
EPS = 1e-6


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one token of plain decode from the 8B's table: launch latency
        {"name": "embed token", "op": "embed", "M": 1, "N": 151936, "K": 4096, "scale": 1.0},
        # a chunk of prompts, frequent tokens repeated, idle slots among them: memory bound
        {"name": "embed prompt", "op": "embed", "M": 8191, "N": 151936, "K": 4096, "scale": 1.0},
        # one new token for each of 48 sequences, contexts up to the model's longest, slots without a sequence
        {"name": "rotate tokens", "op": "rotate", "seqs": 48, "context": 131072, "new": 1, "q_heads": 32, "heads": 8,
         "dim": 128, "norm": True, "rot": 128, "idle": 2},
        # three ragged prompts: memory bound
        {"name": "rotate prompts", "op": "rotate", "seqs": 3, "context": 4096, "new": 2047, "q_heads": 32, "heads": 8,
         "dim": 128, "norm": True, "rot": 128, "idle": 0},
        # one token through the 8B's gate and up projections: weights from memory
        {"name": "gated token", "op": "linear", "M": 1, "N": 12288, "K": 4096, "gate": True, "act": "silu", "bias": False,
         "res": False},
        # a few rows of odd sizes with every part of the epilogue
        {"name": "linear odd", "op": "linear", "M": 11, "N": 1003, "K": 1019, "gate": True, "act": "gelu", "bias": True,
         "res": True},
        # seven drafted tokens and the one before them
        {"name": "gated drafted", "op": "linear", "M": 8, "N": 12288, "K": 4096, "gate": True, "act": "silu",
         "bias": False, "res": False},
        # a prompt chunk through the down projection, back onto the residual stream
        {"name": "residual prompt", "op": "linear", "M": 512, "N": 4096, "K": 12288, "gate": False, "act": "none",
         "bias": False, "res": True},
        # a long prompt through gate and up: matrix bound
        {"name": "gated prompt", "op": "linear", "M": 2048, "N": 12288, "K": 4096, "gate": True, "act": "silu",
         "bias": False, "res": False},
        # a serving step: places for eight drafted tokens of 256 sequences, 32 of them branched since their last one
        {"name": "pages step", "op": "pages", "kind": "step", "seqs": 256, "context": 8192, "new": 8, "twins": 32,
         "spare": 1024, "heads": 8, "dim": 128, "page": 64, "layers": 0},
        # one prompt branched into eight answers: pages shared, the part-filled one copied in every layer
        {"name": "pages fork", "op": "pages", "kind": "fork", "seqs": 8, "context": 4099, "new": 1, "twins": 0,
         "spare": 15, "heads": 8, "dim": 128, "page": 64, "layers": 36},
        # half of a batch has ended: its pages freed, the others' moved together
        {"name": "pages compact", "op": "pages", "kind": "compact", "seqs": 24, "context": 2047, "new": 0, "twins": 4,
         "spare": 33, "heads": 8, "dim": 128, "page": 64, "layers": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "rotate", "linear", "linear", "pages"])
    if op == "embed":
        K = _log(rng, 64, 8192)
        return {"op": op, "M": _log(rng, 1, min(8191, 8191 * 4096 // K)), "N": _log(rng, 2, 200000), "K": K,
                "scale": rng.choice([1.0, math.sqrt(K)])}
    if op == "rotate":
        heads, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([64, 128])
        new = rng.choice([1, 1, rng.randint(2, 16), _log(rng, 16, 2047)])
        seqs = max(1, min(_log(rng, 1, 64), 3 * 2047 * 40 // (new * heads * (group + 1))))
        return {"op": op, "seqs": seqs, "context": max(new, _log(rng, 1, 131072)), "new": new, "q_heads": heads * group,
                "heads": heads, "dim": dim, "norm": rng.random() < 0.7, "rot": rng.choice([dim, dim, dim // 2]),
                "idle": rng.choice([0, 1])}
    if op == "linear":
        case = {"op": op, "M": rng.choice([1, rng.randint(2, 16), _log(rng, 17, 2048)]), "N": _log(rng, 16, 16384),
                "K": _log(rng, 64, 16384), "gate": rng.random() < 0.5, "act": rng.choice(["none", "silu", "gelu"]),
                "bias": rng.random() < 0.4, "res": rng.random() < 0.4}
        if rng.random() < 0.5:  # as in most models; the others odd
            case["N"], case["K"] = -(-case["N"] // 64) * 64, -(-case["K"] // 64) * 64
        top = max(work(c)["flops"] for c in listed())
        while work(case)["flops"] > top:
            case["M"] = max(1, case["M"] * 2 // 3)
        return case
    kind, page = rng.choice(["step", "fork", "compact"]), rng.choice([16, 32, 64, 128])
    case = {"op": op, "kind": kind, "heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128]), "page": page}
    if kind == "step":
        # with few spare pages the last sequences get none
        case.update(seqs=_log(rng, 1, 256), context=_log(rng, 1, 8192), new=_log(rng, 1, 64), layers=0,
                    spare=rng.choice([0, 5, 64, 1024]))
        case["twins"] = rng.randint(0, case["seqs"] // 2)
    else:
        case.update(seqs=_log(rng, 1, 24), context=_log(rng, 1, 4099 if kind == "fork" else 2047), twins=0,
                    new=1 if kind == "fork" else 0, layers=rng.randint(1, 8), spare=rng.randint(32, 64))
        if kind == "compact":
            case["twins"] = rng.randint(0, case["seqs"] // 2)
    return case


def _sequences(case):
    """New and total tokens of each sequence: ragged, the first the longest, a function of the case alone."""
    r = random.Random("%(seqs)d %(context)d %(new)d" % case)
    new = [case["new"]] + [r.randint((case["new"] + 1) // 2, case["new"]) for _ in range(case["seqs"] - 1)]
    total = [case["context"]] + [max(n, r.randint(1, case["context"])) for n in new[1:]]
    idle = case.get("idle", 0)  # slots of a fixed batch that hold no sequence: one row, no tokens
    return new + [1] * idle, total + [0] * idle


def _held(case):
    """(tokens held, tokens wanted or kept) of each row of the page table, a function of the case alone."""
    if case["kind"] == "fork":  # row 0 holds the prompt, the others branch from it
        return [case["context"]] * (case["seqs"] + 1), [case["context"] + 1] * (case["seqs"] + 1)
    r = random.Random("%(seqs)d %(context)d %(twins)d" % case)
    held = [case["context"]] + [r.randint(1, case["context"]) for _ in range(case["seqs"] - 1)]
    for i in range(case["twins"]):  # the last ones hold the same pages as the first
        held[-1 - i] = held[i]
    if case["kind"] == "step":
        return held, [h + r.randint((case["new"] + 1) // 2, case["new"]) for h in held]
    # every other one has ended; some others lose what was drafted past their end
    return held, [0 if i % 2 else max(0, h - r.choice([0, 0, 5])) for i, h in enumerate(held)]


def work(case):
    if case["op"] == "embed":
        n = case["M"] * case["K"]
        return {"bytes": 5 * n + 8 * case["M"], "flops": 2 * n}
    if case["op"] == "rotate":
        new, _ = _sequences(case)
        n = sum(new) * (case["q_heads"] + case["heads"]) * case["dim"]
        return {"bytes": 8 * n, "flops": 8 * n}
    if case["op"] == "linear":
        M, N, K, mats = case["M"], case["N"], case["K"], 1 + case["gate"]
        return {"bytes": mats * N * (16 * -(-K // 64) + 8 + 4 * case["bias"]) + M * (K + 8) + 4 * M * N * (1 + case["res"]),
                "flops": 2 * M * N * K * mats}
    held, want = _held(case)
    P, S, pages, J = case["page"], len(held), _pages(case), _columns(case)
    bytes_page = 2 * case["heads"] * (P * case["dim"] + 4)
    small = 4 * pages + 20 * S
    if case["kind"] == "step":
        return {"bytes": small + 4 * sum(-(-w // P) - -(-h // P) for h, w in zip(held, want)), "flops": pages}
    if case["kind"] == "fork":
        copied = case["seqs"] if case["context"] % P else 0
        small += 4 * (S - 1) * -(-case["context"] // P)
    else:
        live = sum(-(-w // P) for w in want)
        copied = live * (pages - min(pages, live)) // pages  # pages in use behind the place where the last one ends up
        small += 4 * S * J
    return {"bytes": small + 2 * copied * bytes_page * case["layers"], "flops": pages}


def _columns(case):
    return -(-(case["context"] + case["new"]) // case["page"]) + 1


def _pages(case):
    held, _ = _held(case)
    rows = held[:1] if case["kind"] == "fork" else held[: len(held) - case["twins"]]
    return sum(-(-h // case["page"]) for h in rows) + case["spare"]


# ------------------------------------------------------------------ inputs --

def _ternary(g, N, K):
    """Packed rows of random states (62.6 % zeros), their scales and sums."""
    ld = 16 * -(-K // 64)
    w = torch.ones(N, 4 * ld, dtype=torch.uint8, device=DEV)  # codes: state + 1
    u = torch.rand(N, K, generator=g, device=DEV)
    w[:, :K] = torch.where(u < 0.626, 1, torch.where(u < 0.813, 0, 2)).to(torch.uint8)
    rowsum = w.to(torch.int32).sum(1, dtype=torch.int32) - 4 * ld
    w = w.reshape(N, ld // 4, 4, 4)  # word, weights 4k .. 4k + 3 of it at bit 2k, byte
    packed = (w[:, :, 0] | w[:, :, 1] << 2 | w[:, :, 2] << 4 | w[:, :, 3] << 6).reshape(N, ld).contiguous()
    return packed, 0.01 + 0.09 * torch.rand(N, generator=g, device=DEV), rowsum


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    normal = lambda *n: torch.randn(*n, generator=g, device=DEV)  # noqa: E731
    if case["op"] == "embed":
        M, N, K = case["M"], case["N"], case["K"]
        ld = -(-K // 16) * 16
        s["W"] = torch.randint(-127, 128, (N, ld), generator=g, device=DEV, dtype=torch.int8)
        s["s_row"] = 0.001 + 0.009 * torch.rand(N, generator=g, device=DEV)
        # frequent tokens come often; -1 stands in slots without a token
        ids = (N ** torch.rand(M, generator=g, device=DEV, dtype=torch.float64)).long().clamp(max=N) - 1
        ids[::97][1:] = -1
        s["ids"] = ids.to(torch.int32)
        s["x"] = torch.empty(M, K, device=DEV)
        return s
    if case["op"] == "rotate":
        new, total = _sequences(case)
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        Hq, H, D, R = case["q_heads"], case["heads"], case["dim"], case["rot"]
        s["rows"], s["max_new"] = start[-1], max(new)
        s["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        s["len"] = torch.tensor(total, dtype=torch.int32, device=DEV)
        s["q"], s["k"] = 3 * normal(s["rows"], Hq * D), 3 * normal(s["rows"], H * D)
        s["k"][:, :: 61] *= 6  # keys have channels far larger than the others
        s["q_gain"] = 0.5 + torch.rand(D, generator=g, device=DEV) if case["norm"] else None
        s["k_gain"] = 0.5 + torch.rand(D, generator=g, device=DEV) if case["norm"] else None
        s["inv_freq"] = (1e6 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)).float()
        # rows without a place are left as they were
        s["q_out"], s["k_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
        if own:
            from packed_bit_gemv_tern_amd import tern
            s["batch"] = tern.make_kv_batch(None, 0, s["start"], s["len"], len(new), s["rows"], s["max_new"])
        return s
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        ldq = -(-K // 16) * 16
        s["q"] = torch.randint(-128, 128, (M, ldq), generator=g, device=DEV, dtype=torch.int8)
        # activations of about 1, sums over K of a few units where no scale follows
        s["s_act"] = (0.5 + torch.rand(M, generator=g, device=DEV)) * (0.3 / math.sqrt(K))
        s["z"] = torch.randint(-8, 9, (M,), generator=g, device=DEV, dtype=torch.int32)
        s["w"] = _ternary(g, N, K) + (normal(N) if case["bias"] else None,)
        s["up"] = _ternary(g, N, K) + (normal(N) if case["bias"] else None,) if case["gate"] else None
        s["res"] = normal(M, N) if case["res"] else None
        s["y"] = torch.empty(M, N, device=DEV)
        if own:
            from packed_bit_gemv_tern_amd import tern
            s["weights"] = tern.make_weights(*s["w"])
            s["up_weights"] = tern.make_weights(*s["up"]) if case["gate"] else None
        return s
    held, want = _held(case)
    S, J, P, H, D, pages = len(held), _columns(case), case["page"], case["heads"], case["dim"], _pages(case)
    length = torch.tensor(held, device=DEV)
    rows = 1 if case["kind"] == "fork" else S - case["twins"]
    table = torch.full((S, J), -1, dtype=torch.int64, device=DEV)
    holds = torch.arange(J, device=DEV) < ((length + P - 1) // P)[:, None]
    holds[rows:] = False
    place = torch.randperm(pages, generator=g, device=DEV)
    table[holds] = place[: int(holds.sum())]
    if case["twins"]:
        table[rows:] = table[: case["twins"]].flip(0)
    refs = torch.bincount(table[table >= 0], minlength=pages)
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    s["first_table"], s["first_refs"] = i32(table), i32(refs)
    s["table"], s["refs"] = i32(table), i32(refs)
    s["len"], s["want"] = i32(length), torch.tensor(want, dtype=torch.int32, device=DEV)
    s["granted"] = torch.empty(S, dtype=torch.int32, device=DEV)
    moves = pages // 2 if case["kind"] == "compact" else S
    s["from"], s["to"] = (torch.empty(moves, dtype=torch.int32, device=DEV) for _ in range(2))
    s["live"] = torch.empty(1, dtype=torch.int32, device=DEV)
    L = case["layers"]
    if L:
        for name in ("k", "v"):
            shape = (L, pages, H, P, D) if name == "k" else (L, pages, H, D, P)
            s[name] = torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)
            s[name + "_scale"] = 0.005 + 0.02 * torch.rand(L, pages, H, generator=g, device=DEV)
    if case["kind"] == "fork":
        s["src"] = torch.zeros(S - 1, dtype=torch.int32, device=DEV)
        s["dst"] = torch.arange(1, S, dtype=torch.int32, device=DEV)
    if own:
        from packed_bit_gemv_tern_amd import tern
        s["pool"] = tern.make_kv_pool(s["refs"], s["table"], J, S, pages, P)
        s["workspace"] = torch.empty(tern.tern_kv_pool_workspace_bytes(s["pool"]), dtype=torch.uint8, device=DEV)
        if L:
            s["layers"] = tern.make_kv_layers([
                tern.make_kv_cache(s["k"][i], s["v"][i], s["k_scale"][i], s["v_scale"][i], pages, H, D, P)
                for i in range(L)])
    return s


# ------------------------------------------------------------- plain forms --

def _plain_embed(s):
    ids, K = s["ids"].long(), s["x"].shape[1]
    at = ids.clamp(min=0)
    x = s["W"][at, :K].float() * s["s_row"][at][:, None] * s["case"]["scale"]
    return torch.where((ids >= 0)[:, None], x, torch.zeros((), device=DEV))


def _plain_rotate(s):
    case, start, total = s["case"], s["start"].long(), s["len"].long()
    D, R = case["dim"], case["rot"]
    row = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(start[1:], row, right=True)
    pos = (total - (start[1:] - start[:-1]))[seq] + row - start[seq]
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = {}
    for name, gain in (("q", s["q_gain"]), ("k", s["k_gain"])):
        x = s[name].reshape(s["rows"], -1, D)
        if gain is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
        a, b = x[..., : R // 2], x[..., R // 2: R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., R:]], -1)
        out[name] = torch.where((pos >= 0)[:, None, None], y, torch.zeros((), device=DEV)).reshape(s["rows"], -1)
    return out


def _states(packed, K):
    """The packed rows' states -1, 0, +1 in 32 bits."""
    word = packed.reshape(packed.shape[0], -1, 1, 4)
    shift = torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=DEV)[:, None]
    return ((word >> shift) & 3).reshape(packed.shape[0], -1)[:, :K].float() - 1


def _plain_linear(s):
    case = s["case"]
    x = s["q"][:, : case["K"]].float() - s["z"].float()[:, None]

    def product(packed, s_row, _, bias):
        y = torch.matmul(x, _states(packed, case["K"]).T) * s_row * s["s_act"][:, None]  # (whole numbers below 2^24)
        return y if bias is None else y + bias

    y = product(*s["w"])
    if case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif case["act"] == "gelu":
        y = y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if case["gate"]:
        y = y * product(*s["up"])
    return y if s["res"] is None else y + s["res"]


def _plain_reserve(s):
    """Pages for the wanted tokens from the lowest free ones, in the order of the sequences."""
    table, refs, length, want, P = s["table"], s["refs"], s["len"].long(), s["want"].long(), s["case"]["page"]
    S, J = table.shape
    row = torch.arange(S, device=DEV)
    j0, j1 = (length + P - 1) // P, (want + P - 1) // P
    grows = (want > length) & (j1 <= J)
    last = table.gather(1, (j0 - 1).clamp(min=0)[:, None])[:, 0].long()  # the page that the next token goes to
    held = refs.long()[last.clamp(min=0)]
    shared = grows & (length % P > 0) & (last >= 0) & (held > 1)
    same = shared[:, None] & shared[None] & (last[:, None] == last[None])
    keeps = shared & (same.sum(1) >= held) & ~(same & (row[None] > row[:, None])).any(1)
    copies = shared & ~keeps
    need = torch.where(grows, j1 - j0, 0) + copies
    upto = torch.cumsum(need, 0)
    granted = ((upto <= (refs <= 0).sum()) | ((need == 0) & ~keeps)) & ((want <= length) | grows)
    place = torch.sort((refs > 0).to(torch.uint8), stable=True)[1]  # the free pages, lowest first
    first = upto - need
    copies &= granted
    to = torch.where(copies, place[first.clamp(max=len(place) - 1)], -1)
    src = torch.where(copies, last, -1)
    at = row[copies]
    refs.index_add_(0, last[copies], torch.full((len(at),), -1, dtype=torch.int32, device=DEV))
    table[at, j0[copies] - 1] = to[copies].to(torch.int32)
    refs[to[copies]] = 1
    j = torch.arange(J, device=DEV)
    fresh = (granted & grows)[:, None] & (j >= j0[:, None]) & (j < j1[:, None])
    ids = place[((first + copies)[:, None] + j - j0[:, None])[fresh]]
    table[fresh] = ids.to(torch.int32)
    refs[ids] = 1
    s["granted"], s["from"], s["to"] = (t.to(torch.int32) for t in (granted, src, to))


def _plain_compact(s):
    """The lowest hole takes the highest page in use, and so on until no hole lies below one."""
    table, refs, length, P = s["table"], s["refs"], s["want"].long(), s["case"]["page"]
    pages, moves = len(refs), s["from"].shape[0]
    page = torch.arange(pages, device=DEV)
    used = refs > 0
    live = used.sum()
    hole, mover = page[~used & (page < live)], page[used & (page >= live)].flip(0)
    n = min(moves, len(hole))
    to = page.clone()
    to[mover[:n]] = hole[:n]
    refs[hole[:n]] = refs[mover[:n]]
    refs[mover[:n]] = 0
    J = table.shape[1]
    holds = (torch.arange(J, device=DEV) < ((length + P - 1) // P)[:, None]) & (table >= 0)
    table[holds] = to[table[holds].long()].to(torch.int32)
    s["from"], s["to"] = (torch.full((moves,), -1, dtype=torch.int32, device=DEV) for _ in range(2))
    s["from"][:n], s["to"][:n] = mover[:n].to(torch.int32), hole[:n].to(torch.int32)
    s["live"] = live.to(torch.int32).reshape(1)


def _plain_pages(s):
    case, table, refs, P = s["case"], s["table"], s["refs"], s["case"]["page"]
    j = torch.arange(table.shape[1], device=DEV)
    pages_of = lambda n: ((n.long() + P - 1) // P)[:, None]  # noqa: E731
    if case["kind"] == "fork":
        rows = table[s["src"].long()]
        rows = torch.where((j < pages_of(s["len"][s["src"].long()])) & (rows >= 0), rows, -1)
        table[s["dst"].long()] = rows
        taken = rows[rows >= 0].long()
        refs.index_add_(0, taken, torch.ones(len(taken), dtype=torch.int32, device=DEV))
    if case["kind"] == "compact":
        gone = (j >= pages_of(s["want"])) & (j < pages_of(s["len"])) & (table >= 0)
        freed = table[gone].long()
        refs.index_add_(0, freed, torch.full((len(freed),), -1, dtype=torch.int32, device=DEV))
        table[gone] = -1
        _plain_compact(s)
    else:
        _plain_reserve(s)
    if case["layers"]:
        there = s["to"] >= 0
        src, to = s["from"][there].long(), s["to"][there].long()
        for name in ("k", "v", "k_scale", "v_scale"):
            s[name][:, to] = s[name][:, src]


# -------------------------------------------------------------------- pass --

def _pages_out(s):
    case = s["case"]
    out = {"table": s["table"], "refs": s["refs"], "from": s["from"], "to": s["to"]}
    out.update({"live": s["live"]} if case["kind"] == "compact" else {"granted": s["granted"]})
    if case["layers"]:  # pages are moved as they are: the codes themselves, whole numbers, and their scales
        out.update({n: s[n] for n in ("k", "v", "k_scale", "v_scale")})
    return out


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "pages":  # the same tables again in every pass
        s["table"].copy_(s["first_table"])
        s["refs"].copy_(s["first_refs"])
    if not own:
        if op == "pages":
            _plain_pages(s)
            return _pages_out(s)
        return {"embed": _plain_embed, "rotate": _plain_rotate, "linear": _plain_linear}[op](s)
    from packed_bit_gemv_tern_amd import tern
    if op == "embed":
        M, K = s["x"].shape
        tern.tern_embed(s["W"], s["s_row"], case["N"], K, s["W"].shape[1], s["ids"], M, s["x"], K, scale=case["scale"])
        return s["x"]
    if op == "rotate":
        D, nq, nk = case["dim"], s["q"].shape[1], s["k"].shape[1]
        tern.tern_qk_norm_rope(s["batch"], D, s["inv_freq"], case["rot"], q=s["q"], ldq=nq, q_heads=case["q_heads"],
                               q_gain=s["q_gain"], q_out=s["q_out"], ldqo=nq, k=s["k"], ldk=nk, heads=case["heads"],
                               k_gain=s["k_gain"], k_out=s["k_out"], ldko=nk, eps=EPS)
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "linear":
        M, N = s["y"].shape
        act = {"none": tern.TERN_ACT_NONE, "silu": tern.TERN_ACT_SILU, "gelu": tern.TERN_ACT_GELU}[case["act"]]
        tern.tern_linear_epilogue(s["weights"], N, case["K"], M, s["q"], s["q"].shape[1], s["s_act"], s["z"], s["y"], N,
                                  up=s["up_weights"], act=act, res=s["res"], ldr=N)
        return s["y"]
    if case["kind"] == "compact":
        tern.tern_kv_truncate(s["pool"], s["len"], s["want"])
        tern.tern_kv_compact(s["pool"], s["want"], s["from"], s["to"], s["from"].shape[0], s["live"], s["workspace"])
    else:
        if case["kind"] == "fork":
            tern.tern_kv_fork(s["pool"], s["len"], s["src"], s["dst"], s["src"].shape[0])
        tern.tern_kv_reserve(s["pool"], s["len"], s["want"], s["granted"], s["from"], s["to"], s["workspace"])
    if case["layers"]:
        tern.tern_kv_copy(s["layers"], s["layers"], s["from"], s["to"], s["from"].shape[0])
    return _pages_out(s)


# ------------------------------------------------------------------- exact --

def _exact_embed(s):
    x = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    there = (s["ids"] >= 0).nonzero()[:, 0]
    at = s["ids"][there].long()
    x[there] = torch.einsum("mk,m->mk", s["W"][at].double()[:, : x.shape[1]], s["s_row"][at].double())
    return x * s["case"]["scale"]


def _exact_rotate(s):
    case = s["case"]
    D, R = case["dim"], case["rot"]
    new, total = _sequences(case)
    pos = torch.cat([torch.arange(t - n, t) for n, t in zip(new, total)]).to(DEV).double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos[:, None] * s["inv_freq"].double())[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].double().reshape(len(pos), -1, D)
        if s[name + "_gain"] is not None:
            x = x * (x.pow(2).sum(-1, keepdim=True) / D + EPS).pow(-0.5) * s[name + "_gain"].double()
        pair = torch.complex(x[..., : R // 2].contiguous(), x[..., R // 2: R].contiguous()) * turn
        y = torch.cat([pair.real, pair.imag, x[..., R:]], -1)
        y[pos < 0] = 0
        out[name] = y.reshape(len(pos), -1)
    return out


def _exact_linear(s):
    case = s["case"]
    K = case["K"]
    a = (s["q"][:, :K].double() - s["z"].double()[:, None]) * s["s_act"].double()[:, None]
    both = []
    for packed, s_row, _, bias in [s["w"]] + ([s["up"]] if case["gate"] else []):
        w = torch.empty(case["N"], 4 * packed.shape[1], dtype=torch.float64, device=DEV)
        for j in range(16):  # weight j of every word of sixteen
            w[:, j::16] = (packed[:, j % 4::4].long() // 4 ** (j // 4) % 4 - 1).double()
        v = a @ w[:, :K].T.contiguous() * s_row.double()
        both.append(v if bias is None else v + bias.double())
    y = both[0]
    if case["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif case["act"] == "gelu":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
        # 1 + tanh cancels for large negative arguments: the same by the sigmoid there
        v = both[0]
        y = torch.where(v < -1, v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)), y)
    for factor in both[1:]:
        y = y * factor
    return y if s["res"] is None else y + s["res"].double()


def _exact_pages(s):
    """Page by page on the host, lists and loops."""
    case, P = s["case"], s["case"]["page"]
    table, refs = s["first_table"].tolist(), s["first_refs"].tolist()
    held, want = _held(case)
    count = lambda n: (n + P - 1) // P  # noqa: E731
    moves, live = [], None
    if case["kind"] == "fork":
        for dst in range(1, len(table)):
            for j in range(count(held[0])):
                table[dst][j] = table[0][j]
                refs[table[0][j]] += 1
    if case["kind"] == "compact":
        for r, row in enumerate(table):
            for j in range(count(want[r]), count(held[r])):
                refs[row[j]] -= 1
                row[j] = -1
        live = sum(n > 0 for n in refs)
        holes = [p for p in range(live) if refs[p] == 0]
        goes = dict(zip(sorted((p for p in range(live, len(refs)) if refs[p]), reverse=True), holes))
        moves = list(goes.items())
        for old, at in moves:
            refs[at], refs[old] = refs[old], 0
        table = [[goes.get(p, p) for p in row] for row in table]
        out = {"live": torch.tensor([live])}
        lists = [m + [-1] * (len(refs) // 2 - len(m)) for m in ([a for a, _ in moves], [b for _, b in moves])]
    else:
        free = [p for p, n in enumerate(refs) if n == 0]
        total, used, granted, pairs = len(free), 0, [], []
        at_page = lambda r: table[r][count(held[r]) - 1] if held[r] % P else -1  # noqa: E731
        first, had = [at_page(r) if want[r] > held[r] else -1 for r in range(len(table))], list(refs)
        for r, row in enumerate(table):
            last = first[r]
            shared = last >= 0 and had[last] > 1
            sole = shared and first.count(last) >= had[last] and last not in first[r + 1:]
            n = count(want[r]) - count(held[r]) + (shared and not sole)
            used += n
            granted.append(int(used <= total or (n == 0 and not sole)))
            pairs.append((-1, -1))
            if not granted[-1]:
                continue
            take = free[used - n: used]
            if shared and not sole:
                pairs[-1] = (last, take[0])
                refs[last] -= 1
                row[count(held[r]) - 1] = take[0]
            row[count(held[r]): count(want[r])] = take[len(take) - (count(want[r]) - count(held[r])):]
            for p in take:
                refs[p] = 1
        out = {"granted": torch.tensor(granted)}
        lists = [[a for a, _ in pairs], [b for _, b in pairs]]
        moves = [p for p in pairs if p[0] >= 0]
    out.update(table=torch.tensor(table), refs=torch.tensor(refs))
    out["from"], out["to"] = (torch.tensor(x) for x in lists)
    if case["layers"]:
        for name in ("k", "v", "k_scale", "v_scale"):
            was, now = s[name], s[name].clone()
            for a, b in moves:
                now[:, b] = was[:, a]
            out[name] = now
    return {n: t.to(DEV) for n, t in out.items()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "rotate": _exact_rotate, "linear": _exact_linear, "pages": _exact_pages}[case["op"]](s)
