"""The decode step's operators between the ternary linears, as measured cases.

Four operators: the RMS norm with the residual's addition and an int8 output
(what every linear and the head read), the append of new keys and values to a
paged int8 cache, the attention over that cache, and the sampling of a token
from the head's logits.  The geometries are the 8B's (hidden 4,096, 32 query
and 8 key/value heads of 128, vocabulary 151,936) and the 0.6B's (hidden
1,024, 16 and 8 heads), with generic ones beside them.
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
        # one token of plain decode, 8B hidden width: launch latency
        {"name": "norm token", "op": "norm", "M": 1, "K": 4096},
        # a small serving batch at an odd width that no vector load divides
        {"name": "norm batch odd", "op": "norm", "M": 37, "K": 1019},
        # a prompt chunk, 8B hidden width: memory bound
        {"name": "norm prompt", "op": "norm", "M": 4096, "K": 4096},
        # one new token for each of 24 sequences after a few tokens, into part-filled pages
        {"name": "append tokens", "op": "append", "seqs": 24, "context": 30, "new": 1, "heads": 8, "dim": 128, "page": 32},
        # three ragged prompts into fresh pages
        {"name": "append prompts", "op": "append", "seqs": 3, "context": 2047, "new": 2047, "heads": 8, "dim": 128,
         "page": 64},
        # one user, one token, a few thousand tokens of context: latency
        {"name": "attend token", "op": "attend", "seqs": 1, "context": 4099, "new": 1, "q_heads": 32, "heads": 8,
         "dim": 128, "page": 64, "idle": 0},
        # seven drafted tokens and the one before them, a long context
        {"name": "attend drafted long", "op": "attend", "seqs": 1, "context": 32771, "new": 8, "q_heads": 32, "heads": 8,
         "dim": 128, "page": 16, "idle": 0},
        # a serving batch of ragged contexts (one slot idle) at the 0.6B's head counts
        {"name": "attend batch", "op": "attend", "seqs": 48, "context": 8192, "new": 1, "q_heads": 16, "heads": 8,
         "dim": 128, "page": 64, "idle": 1},
        # two prompt chunks on top of cached context: matrix bound
        {"name": "attend prompt", "op": "attend", "seqs": 2, "context": 4096, "new": 2048, "q_heads": 32, "heads": 8,
         "dim": 128, "page": 64, "idle": 0},
        # one token, the usual filters, the 8B's vocabulary
        {"name": "sample token", "op": "sample", "M": 1, "N": 151936, "filters": "kp"},
        # eight drafted positions, minimum probability only
        {"name": "sample drafted", "op": "sample", "M": 8, "N": 151936, "filters": "min_p"},
        # a serving batch, every request with its own filters (greedy and unfiltered ones among them)
        {"name": "sample batch", "op": "sample", "M": 96, "N": 151936, "filters": "mixed"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "attend", "attend", "sample"])
    if op == "norm":
        K = _log(rng, 64, 8192)
        return {"op": op, "M": _log(rng, 1, 4096 * 4096 // max(K, 4096)), "K": K}
    if op == "append":
        new = _log(rng, 1, 1024)
        return {"op": op, "seqs": max(1, min(_log(rng, 1, 48), 4096 // new)), "context": new + rng.randint(0, 96),
                "new": new, "heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128]),
                "page": rng.choice([16, 32, 64, 128])}
    if op == "attend":
        heads, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([64, 128])
        case = {"op": op, "new": rng.choice([1, 1, rng.randint(2, 16), _log(rng, 16, 1024)]), "q_heads": heads * group,
                "heads": heads, "dim": dim, "page": rng.choice([16, 32, 64, 128]), "idle": rng.choice([0, 1])}
        case["context"] = max(case["new"], _log(rng, 1, 32768))
        # no more keys and values are read, and no more work is done, than in the largest listed cases
        room = min(48 * 8192 * 8 // (case["context"] * heads), 64)
        case["seqs"] = _log(rng, 1, max(1, room))
        while _cost(case) > max(_cost(c) for c in listed()):
            case["seqs"], case["new"] = max(1, case["seqs"] // 2), max(1, case["new"] * 2 // 3)
        return case
    N = _log(rng, 2, 200000)
    return {"op": op, "M": _log(rng, 1, max(1, min(256, 96 * 151936 // N))), "N": N,
            "filters": rng.choice(["none", "k", "p", "kp", "min_p", "mixed"])}


def _sequences(case):
    """New and total tokens of each sequence: ragged, the first the longest, a function of the case alone."""
    r = random.Random("%(seqs)d %(context)d %(new)d" % case)
    new = [case["new"]] + [r.randint((case["new"] + 1) // 2, case["new"]) for _ in range(case["seqs"] - 1)]
    total = [case["context"]] + [max(n, r.randint(1, case["context"])) for n in new[1:]]
    idle = case.get("idle", 0)  # slots of a fixed batch that hold no sequence: one row, no tokens
    return new + [1] * idle, total + [0] * idle


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def work(case):
    if case["op"] == "norm":
        n = case["M"] * case["K"]
        return {"bytes": 13 * n + 4 * case["K"] + 8 * case["M"], "flops": 10 * n}
    if case["op"] == "sample":
        return {"bytes": 4 * case["M"] * case["N"] + 32 * case["M"], "flops": 4 * case["M"] * case["N"]}
    new, total = _sequences(case)
    P, H, D = case["page"], case["heads"], case["dim"]
    pages = sum(-(-t // P) for t in total)
    if case["op"] == "append":
        n = 2 * sum(new) * H * D
        return {"bytes": 5 * n + 16 * pages * H + 4 * pages, "flops": 4 * n}
    seen = sum(sum(range(max(0, t - n) + 1, t + 1)) for n, t in zip(new, total))
    return {"bytes": 2 * sum(total) * H * D + 8 * pages * H + 4 * pages + 8 * sum(new) * case["q_heads"] * D,
            "flops": 4 * case["q_heads"] * D * seen}


# ------------------------------------------------------------------ inputs --

def _hidden(g, M, K):
    """A residual stream's rows: normal, with a few outlier channels."""
    x = torch.randn(M, K, generator=g, device=DEV)
    x[:, :: 256] *= 20
    return x


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        s["x"], s["res"] = torch.randn(M, K, generator=g, device=DEV), _hidden(g, M, K)
        s["gain"] = 0.5 + torch.rand(K, generator=g, device=DEV)
        ldq = -(-K // 16) * 16
        s["h"] = torch.empty(M, K, device=DEV)
        s["q"] = torch.empty(M, ldq, dtype=torch.int8, device=DEV)
        s["s_act"] = torch.empty(M, device=DEV)
        s["z"] = torch.empty(M, dtype=torch.int32, device=DEV)
        return s
    if case["op"] == "sample":
        M, N = case["M"], case["N"]
        # logits of a peaked distribution: a wide bulk and some hundreds of likely tokens
        x = 2.2 * torch.randn(M, N, generator=g, device=DEV)
        likely = torch.rand(M, N, generator=g, device=DEV) < 200 / N
        x = torch.where(likely, 4 + 10 * torch.rand(M, N, generator=g, device=DEV), x)
        s["logits"] = x
        s["u"] = torch.rand(M, generator=g, device=DEV)
        uni = lambda lo, hi: lo + (hi - lo) * torch.rand(M, generator=g, device=DEV)  # noqa: E731
        row = torch.arange(M, device=DEV)
        f = case["filters"]
        s["temperature"] = uni(0.4, 1.2)
        s["top_k"] = torch.randint(1, 200, (M,), generator=g, device=DEV, dtype=torch.int32) if f in ("k", "kp", "mixed") else None
        s["top_p"] = uni(0.5, 0.99) if f in ("p", "kp", "mixed") else None
        s["min_p"] = uni(0.01, 0.2) if f in ("min_p", "mixed") else None
        if f == "mixed":  # row by row: which filters a request has, some none, some greedy
            s["top_k"] = torch.where(row % 2 == 0, s["top_k"], 0)
            s["top_p"] = torch.where(row % 3 != 1, s["top_p"], 1.0)
            s["min_p"] = torch.where(row % 5 == 2, s["min_p"], 0.0)
            s["temperature"] = torch.where(row % 7 == 3, 0.0, s["temperature"])
        s["token"] = torch.empty(M, dtype=torch.int32, device=DEV)
        s["prob"] = torch.empty(M, device=DEV)
        s["kept"] = torch.empty(M, dtype=torch.int32, device=DEV)
        if own:
            from packed_bit_gemv_tern_amd import tern
            s["workspace"] = torch.empty(tern.tern_sample_workspace_bytes(M, N), dtype=torch.uint8, device=DEV)
        return s
    new, total = _sequences(case)
    S, H, D, P = len(new), case["heads"], case["dim"], case["page"]
    J = max(1, -(-max(total) // P))
    pages = S * J
    # what the cache holds already, in every slot: codes of normal values, another scale for each page and head
    for name, shape in (("k", (pages, H, P, D)), ("v", (pages, H, D, P))):
        codes = torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)
        s[name + "_codes"] = codes
        s[name + "_scale"] = 0.005 + 0.02 * torch.rand(pages, H, generator=g, device=DEV)
    s["table"] = torch.randperm(pages, generator=g, device=DEV).reshape(S, J).to(torch.int32)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s["rows"], s["max_new"], s["max_len"] = start[-1], max(new), max(total)
    s["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
    s["len"] = torch.tensor(total, dtype=torch.int32, device=DEV)
    if case["op"] == "append":
        # keys have channels far larger than the others, values do not
        s["k_new"] = torch.randn(s["rows"], H * D, generator=g, device=DEV)
        s["k_new"][:, :: 61] *= 6
        s["v_new"] = torch.randn(s["rows"], H * D, generator=g, device=DEV)
    else:
        s["q"] = 3.0 * torch.randn(s["rows"], case["q_heads"] * D, generator=g, device=DEV)
        s["scale"] = D ** -0.5
        s["y"] = torch.empty_like(s["q"])
    if own:
        from packed_bit_gemv_tern_amd import tern
        s["cache"] = tern.make_kv_cache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], pages, H, D, P)
        s["batch"] = tern.make_kv_batch(s["table"], J, s["start"], s["len"], S, s["rows"], s["max_new"], s["max_len"])
        if case["op"] == "attend":
            n = tern.tern_attention_workspace_bytes(s["cache"], s["batch"], case["q_heads"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------- plain forms --

def _quantised(y):
    """(codes, scale, zero point) of each row: its range widened to hold zero, in 255 steps."""
    lo, hi = y.amin(-1, keepdim=True).clamp(max=0), y.amax(-1, keepdim=True).clamp(min=0)
    s = (hi - lo) / torch.full((), 255.0, device=y.device)
    s = torch.where(hi == lo, torch.ones_like(s), s)
    z = -128 - torch.round(lo / s)
    return (torch.round(y / s) + z).clamp(-128, 127), s, z


def _plain_norm(s):
    h = s["x"] + s["res"]
    d = h.double()
    y = (d / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS) * s["gain"].double()).float()
    q, scale, z = _quantised(y)
    return {"h": h, "values": (q - z) * scale, "s_act": scale[:, 0], "z": z[:, 0].to(torch.int32)}


def _plain_append(s):
    case, start, total = s["case"], s["start"].long(), s["len"].long()
    H, D, P = case["heads"], case["dim"], case["page"]
    S, J = s["table"].shape
    n = start[1:] - start[:-1]
    row = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(start[1:], row, right=True)
    pos = (total - n)[seq] + row - start[seq]
    first = (total - n) // P  # the first page of a sequence that gets tokens
    C = (s["max_new"] + P - 2) // P + 1  # pages that one sequence's tokens can touch
    page = first[:, None] + torch.arange(C, device=DEV)
    touched = page <= ((total - 1) // P)[:, None]
    ids = s["table"].long().gather(1, page.clamp(max=J - 1))
    held = ((total - n)[:, None] - page * P).clamp(0, P)  # tokens that a page holds already
    old = torch.arange(P, device=DEV) < held[:, :, None]
    out = {}
    for name, new in (("k", s["k_new"]), ("v", s["v_new"])):
        codes, scale = s[name + "_codes"], s[name + "_scale"]
        x = torch.zeros(S, C, P, H, D, device=DEV)
        fresh = torch.zeros(S, C, P, dtype=torch.bool, device=DEV)
        x[seq, pos // P - first[seq], pos % P] = new.reshape(-1, H, D)
        fresh[seq, pos // P - first[seq], pos % P] = True
        x = x.permute(0, 1, 3, 2, 4)  # S, C, H, P, D
        was = torch.where(held[:, :, None] > 0, scale[ids], torch.zeros((), device=DEV))
        now = torch.maximum(was, x.abs().amax((-1, -2)) / torch.full((), 127.0, device=DEV))
        ratio = torch.where(now > 0, was / now, torch.ones_like(now))[..., None, None]
        c = codes[ids] if name == "k" else codes[ids].transpose(-1, -2)
        c = torch.where(old[:, :, None, :, None], torch.round(c.float() * ratio), c.float())
        q = torch.round(x / torch.where(now > 0, now, torch.ones_like(now))[..., None, None]).clamp(-127, 127)
        c = torch.where(fresh[:, :, None, :, None], q, c).to(torch.int8)
        c = c if name == "k" else c.transpose(-1, -2)
        codes[ids[touched]] = c[touched]
        scale[ids[touched]] = now[touched]
        out[name] = codes * scale[:, :, None, None]
        out[name + "_scale"] = scale
    return out


def _plain_attend(s):
    case, start, total = s["case"], s["start"].long(), s["len"].long()
    Hq, H, D, P = case["q_heads"], case["heads"], case["dim"], case["page"]
    S, J = s["table"].shape
    G, n, T = Hq // H, start[1:] - start[:-1], s["max_new"]
    ids = s["table"].long()
    k = s["k_codes"][ids].float() * s["k_scale"][ids][..., None, None]  # S, J, H, P, D
    v = s["v_codes"][ids].float() * s["v_scale"][ids][..., None, None]  # S, J, H, D, P
    k = k.permute(0, 2, 4, 1, 3).reshape(S, H, D, J * P)
    v = v.permute(0, 2, 1, 4, 3).reshape(S, H, J * P, D)
    t = torch.arange(T, device=DEV)
    rows = (start[:-1, None] + t).clamp(max=s["rows"] - 1)
    q = s["q"][rows].reshape(S, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, T * G, D)
    a = torch.matmul(q, k) * s["scale"]
    pos = (total - n)[:, None] + t  # a row's own position
    seen = torch.arange(J * P, device=DEV) <= pos[:, :, None]
    seen = seen.repeat_interleave(G, 1)[:, None]
    a = a.masked_fill(~seen, -math.inf)
    m = a.amax(-1, keepdim=True)
    e = torch.exp(a - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    y = torch.matmul(e, v) / e.sum(-1, keepdim=True).clamp(min=1e-30)
    y = y.reshape(S, H, T, G, D).permute(0, 2, 1, 3, 4).reshape(S, T, Hq * D)
    return y[t < n[:, None]]


def _plain_sample(s):
    x = s["logits"]
    x = torch.where(torch.isnan(x), -math.inf, x).double()
    mx = x.amax(-1, keepdim=True)
    T = s["temperature"].double()[:, None]
    w = torch.exp((x - mx) / T)
    w = torch.where((T > 0) & (x < mx), w, (x == mx).double())
    w = torch.where((x > -math.inf) & ((T > 0) | (x == mx)), w, 0.0)
    v, order = torch.sort(x, stable=True, dim=-1, descending=True)
    ws = w.gather(1, order)
    rank = torch.arange(x.shape[1], device=x.device)
    keep = (v > -math.inf) & ((T > 0) | (rank == 0))
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep &= (k <= 0) | (rank < k)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        wk = ws * keep
        run = torch.cumsum(wk, -1)
        keep &= (p >= 1) | (run - wk < p * run[:, -1:]) | (rank == 0)
    if s["min_p"] is not None:
        keep &= (ws >= s["min_p"].double()[:, None]) | (rank == 0)
    kept = torch.zeros_like(keep).scatter(1, order, keep)
    run = torch.cumsum(w * kept, -1)
    token = (run <= s["u"].double()[:, None] * run[:, -1:]).sum(-1, keepdim=True)
    prob = w.gather(1, token) / run[:, -1:]
    return {"token": token[:, 0].to(torch.int32), "prob": prob[:, 0].float(), "kept": keep.sum(-1).to(torch.int32)}


# -------------------------------------------------------------------- pass --

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}[op](s)
    from packed_bit_gemv_tern_amd import tern
    if op == "norm":
        M, K = s["x"].shape
        tern.tern_rmsnorm_quantize(s["x"], s["gain"], EPS, M, K, K, s["q"], s["q"].shape[1], s["s_act"], s["z"],
                                   res=s["res"], ldr=K, h=s["h"], ldh=K)
        values = (s["q"][:, :K] - s["z"][:, None]) * s["s_act"][:, None]
        return {"h": s["h"], "values": values, "s_act": s["s_act"], "z": s["z"]}
    if op == "append":
        ld = s["k_new"].shape[1]
        tern.tern_kv_append(s["cache"], s["batch"], s["k_new"], ld, s["v_new"], ld)
        return {"k": s["k_codes"] * s["k_scale"][:, :, None, None], "k_scale": s["k_scale"],
                "v": s["v_codes"] * s["v_scale"][:, :, None, None], "v_scale": s["v_scale"]}
    if op == "attend":
        ld = s["q"].shape[1]
        tern.tern_attention(s["cache"], s["batch"], s["q"], ld, s["case"]["q_heads"], s["scale"], s["y"], ld,
                            s["workspace"])
        return s["y"]
    M, N = s["logits"].shape
    tern.tern_sample(s["logits"], M, N, N, s["temperature"], s["u"], s["token"], s["workspace"], top_k=s["top_k"],
                     top_p=s["top_p"], min_p=s["min_p"], prob=s["prob"], kept=s["kept"])
    return {"token": s["token"], "prob": s["prob"], "kept": s["kept"]}


# ------------------------------------------------------------------- exact --

def _exact_norm(s):
    h = (s["x"].double() + s["res"].double()).float()  # the sum is held in 32 bits
    d = h.double()
    r = (d.pow(2).sum(1) / d.shape[1] + EPS).pow(-0.5)
    y = torch.einsum("mk,m,k->mk", d, r, s["gain"].double()).float()
    lo, hi = torch.clamp(y.min(1).values, max=0), torch.clamp(y.max(1).values, min=0)
    # scale and codes are 32-bit and 8-bit numbers by definition: each step rounded from 64 bits
    scale = ((hi.double() - lo.double()).float().double() / 255).float().double()
    scale = torch.where(hi == lo, torch.ones_like(scale), scale)
    z = -128 - (lo.double() / scale).float().double().round()
    q = (y.double() / scale[:, None]).float().double().round() + z[:, None]
    return {"h": s["x"].double() + s["res"].double(), "values": (q.clamp(-128, 127) - z[:, None]) * scale[:, None],
            "s_act": scale, "z": None}


def _exact_append(s):
    """Token by token of the definition, over pages: in 64 bits, each rounding that the format makes written out."""
    case = s["case"]
    H, D, P = case["heads"], case["dim"], case["page"]
    new, total = _sequences(case)
    table, out, at = s["table"].tolist(), {}, [0]
    for n in new:
        at.append(at[-1] + n)
    for name in ("k", "v"):
        codes, scale = s[name + "_codes"].double().cpu(), s[name + "_scale"].double().cpu()
        x = s[name + "_new"].double().cpu().reshape(-1, H, D)
        for i, (n, t) in enumerate(zip(new, total)):
            for j in range((t - n) // P, (t - 1) // P + 1):
                lo, hi = max(t - n, j * P), min(t, (j + 1) * P)
                part = x[at[i] + lo - (t - n): at[i] + hi - (t - n)].permute(1, 0, 2)  # H, tokens, D
                c = codes[table[i][j]] if name == "k" else codes[table[i][j]].transpose(1, 2)
                held = lo - j * P
                was = scale[table[i][j]].clone() if held else torch.zeros(H, dtype=torch.float64)
                now = torch.maximum(was, (part.abs().amax((1, 2)) / 127).float().double())
                ratio = (was / now).float().double()[:, None, None]
                c[:, :held] = (c[:, :held] * ratio).float().double().round()
                c[:, held: hi - j * P] = (part / now[:, None, None]).float().double().round().clamp(-127, 127)
                scale[table[i][j]] = now
        out[name], out[name + "_scale"] = codes * scale[:, :, None, None], scale
    return out


def _exact_attend(s):
    case = s["case"]
    Hq, H, D, P = case["q_heads"], case["heads"], case["dim"], case["page"]
    new, total = _sequences(case)
    y = torch.zeros(s["rows"], H, Hq // H, D, dtype=torch.float64, device=DEV)
    q = s["q"].double().reshape(s["rows"], H, Hq // H, D)
    at = 0
    for i, (n, t) in enumerate(zip(new, total)):
        if t:
            ids = s["table"][i, : -(-t // P)].long()
            k = s["k_codes"][ids].double() * s["k_scale"][ids].double()[:, :, None, None]
            v = s["v_codes"][ids].double() * s["v_scale"][ids].double()[:, :, None, None]
            for h in range(H):
                kh, vh = k[:, h].reshape(-1, D)[:t], v[:, h].transpose(1, 2).reshape(-1, D)[:t]
                a = q[at: at + n, h].reshape(-1, D) @ kh.T.contiguous() * s["scale"]
                own_place = torch.arange(t - n, t, device=DEV).repeat_interleave(Hq // H)
                a[torch.arange(t, device=DEV)[None] > own_place[:, None]] = -math.inf
                y[at: at + n, h] = (torch.softmax(a, 1) @ vh).reshape(n, -1, D)
        at += n
    return y.reshape(s["rows"], -1)


def _exact_sample(s):
    """The chosen token's probability, row by row; the whole numbers beside it have no other value in 64 bits."""
    prob = []
    for i, x in enumerate(s["logits"].double()):
        T, u = float(s["temperature"][i]), float(s["u"][i])
        if T <= 0:
            prob.append(1.0)
            continue
        w = torch.exp((x - x.max()) / T)
        w, order = torch.sort(w / w.sum(), stable=True, dim=0, descending=True)
        k = int(s["top_k"][i]) if s["top_k"] is not None else 0
        n = min(k, len(w)) if k > 0 else len(w)
        p = float(s["top_p"][i]) if s["top_p"] is not None else 1.0
        run = torch.cumsum(w[:n], 0)
        if p < 1:
            n = min(n, 1 + int((run[:-1] < p * run[-1]).sum()))
        if s["min_p"] is not None:
            n = min(n, max(1, int((w >= float(s["min_p"][i]) * w[0]).sum())))
        at, back = torch.sort(order[:n])
        mass = w[:n][back]
        run = torch.cumsum(mass, 0)
        chosen = min(n - 1, int((run <= u * run[-1]).sum()))
        prob.append(float(mass[chosen] / run[-1]))
    return {"token": None, "prob": torch.tensor(prob, dtype=torch.float64), "kept": None}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](s)
