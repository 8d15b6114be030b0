"""The operators around a decoder's mixture-of-experts layer, as measured cases.

Three operators that a decoder layer runs beside the routed experts:

- ``norm``    r = x + s * gate * rms(o; w_post),  h = rms(r; w_pre): the norms after one
              block and before the next, with the block's gate and residual scale;
- ``append``  rotate a token's queries and keys by its position, write keys and
              values into a paged cache (bf16, or e4m3 with a scale per key-value head);
- ``attend``  attention of one new token per sequence over the paged cache.

``run`` computes them in elementary torch operations, or, where ``own`` is true,
through the package's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _attend(B, Hq, Hkv, D, page, max_len, lens="ragged", cache="bf16", window=0, softcap=0.0, layout="hnd"):
    return dict(op="attend", B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, max_len=max_len, lens=lens, cache=cache,
                window=window, softcap=softcap, layout=layout)


def _append(T, seqs, Hq, Hkv, D, page, far, cache="bf16", rotary=None, interleaved=False, layout="hnd"):
    return dict(op="append", T=T, seqs=seqs, Hq=Hq, Hkv=Hkv, D=D, page=page, far=far, cache=cache,
                rotary=D if rotary is None else rotary, interleaved=interleaved, layout=layout)


def _norm(T, H, res="f32", o="bf16", h="bf16", post=True, gate="none", scale=1.0, offset=0.0):
    return dict(op="norm", T=T, H=H, res=res, o=o, h=h, post=post, gate=gate, scale=scale, offset=offset)


def listed():
    return [
        # the first tokens of a conversation on a 512-wide layer (8 heads of 64): pure latency
        dict(_attend(1, 8, 2, 64, 16, 17, "equal"), name="attend_first_tokens"),
        # one user far into a long document, 6144-wide layer (48 heads of 128): the split over the length
        dict(_attend(1, 48, 8, 128, 64, 131072, "equal"), name="attend_one_long"),
        # a serving batch of mixed conversations, some slots idle, small pages
        dict(_attend(64, 48, 8, 128, 16, 16384, "ragged"), name="attend_batch_ragged"),
        # sliding-window layers with capped logits and wide heads, tokens outermost in a page
        dict(_attend(32, 16, 8, 256, 32, 4500, "ragged", window=1024, softcap=50.0, layout="nhd"),
             name="attend_window_cap"),
        # an 8-bit cache under grouped queries, 16 queries to a key-value head
        dict(_attend(48, 64, 4, 128, 64, 9001, "ragged", cache="e4m3"), name="attend_8bit"),
        # one decode token
        dict(_append(1, 1, 48, 8, 128, 64, 5000), name="append_one"),
        # a decode batch into an 8-bit cache, positions up to a million
        dict(_append(61, 61, 48, 8, 128, 16, 1000000, cache="e4m3"), name="append_batch_8bit"),
        # one prefill chunk with half of each head rotated in adjacent pairs
        dict(_append(128, 1, 16, 8, 256, 32, 30000, rotary=128, interleaved=True, layout="nhd"),
             name="append_chunk_partial"),
        # chunks of many sequences at once
        dict(_append(8192, 64, 48, 8, 128, 64, 60000), name="append_many_chunks"),
        # one decode token on the 6144-wide layer
        dict(_norm(1, 6144), name="norm_one"),
        # one prefill chunk on the 2816-wide layer, norms around the block, a gate per channel, 1 + w weights
        dict(_norm(128, 2816, res="bf16", gate="row", scale=0.7, offset=1.0), name="norm_chunk"),
        # many chunks, a gate per token and channel
        dict(_norm(8191, 6144, gate="full", scale=0.25), name="norm_many"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Sizes over the range the listed cases span, odd ones among them."""
    op = rng.choice(("attend", "attend", "append", "norm"))
    if op == "norm":
        H = 64 * _log(rng, 4, 128)
        return _norm(_log(rng, 1, 8191), min(H, 6144), rng.choice(("f32", "bf16")), rng.choice(("f32", "bf16")),
                     rng.choice(("f32", "bf16")), rng.random() < 0.7, rng.choice(("none", "row", "full")),
                     round(rng.uniform(0.1, 1.5), 3), rng.choice((0.0, 1.0)))
    D = rng.choice((64, 128, 256))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    G = rng.choice((1, 2, 4, 5, 6, 8, 12, 16))
    page = rng.choice((16, 32, 48, 64, 128))
    cache = rng.choice(("bf16", "bf16", "e4m3"))
    layout = rng.choice(("hnd", "nhd"))
    if op == "append":
        seqs = _log(rng, 1, 64)
        T = seqs * _log(rng, 1, 110)
        G = min(G, max(1, 40 * 128 // (Hkv * D)))
        return _append(T, seqs, Hkv * G, Hkv, D, page, _log(rng, 200, 1000000), cache,
                       rng.choice((D, D, D // 2, 0)), rng.random() < 0.4, layout)
    B = _log(rng, 1, 64)
    # no more cached values, nor products with them, than the largest listed case has
    lens = rng.choice(("ragged", "equal"))
    most = 64 * 16384 * 8 * 128 * 6 // (B * Hkv * D * max(G, 6) * (3 if lens == "equal" else 1))
    max_len = min(_log(rng, 1, 131072), most)
    return _attend(B, Hkv * G, Hkv, D, page, max_len, lens, cache,
                   rng.choice((0, 0, 0, _log(rng, 1, 4096))), rng.choice((0.0, 0.0, 30.0)), layout)


def _lens(case):
    """Cached tokens of every sequence: a property of the case, so that its work is known."""
    B, L = case["B"], case["max_len"]
    if case["lens"] == "equal":
        return [L] * B
    rng = random.Random(B * 1000003 + L)
    lens = [_log(rng, max(1, L // 16), L) for _ in range(B)]
    lens[rng.randrange(B)] = L
    if B >= 8:
        lens[rng.randrange(1, B)] = 0  # an idle slot
    return lens


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pool(case, n_pages, g, shape_scale):
    """A page pool as [n_pages, Hkv, page, D], its memory in the case's order."""
    Hkv, page, D = case["Hkv"], case["page"], case["D"]
    shape = (n_pages, Hkv, page, D) if case["layout"] == "hnd" else (n_pages, page, Hkv, D)
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    if case["cache"] == "e4m3":
        x = (x * (448 / 5)).clamp_(-448, 448).to(torch.float8_e4m3fn)
    elif shape_scale != 1.0:
        x *= shape_scale
    return x if case["layout"] == "hnd" else x.permute(0, 2, 1, 3)


def _scales(case, seed):
    """What one step of an 8-bit cache stands for, per key-value head (ones for bf16)."""
    rng = random.Random(seed)
    if case["cache"] != "e4m3":
        return torch.ones(case["Hkv"])
    return torch.tensor([rng.uniform(0.5, 1.5) * 5 / 448 for _ in range(case["Hkv"])], dtype=torch.float32)


def _cache(case, st, n_pages, seed, g, max_batch):
    st["k_pages"] = _pool(case, n_pages, g, 1.0)
    st["v_pages"] = _pool(case, n_pages, g, 0.7)
    st["k_scale"], st["v_scale"] = _scales(case, seed + 1), _scales(case, seed + 2)
    rot = case.get("rotary", case["D"])
    st["inv_freq"] = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    st["k_scale_dev"], st["v_scale_dev"] = st["k_scale"].to(DEV), st["v_scale"].to(DEV)
    st["inv_freq_dev"] = st["inv_freq"].to(DEV)
    if own:
        import quantized_routed_expert_moe_gb300 as moe
        e4m3 = case["cache"] == "e4m3"
        st["kv"] = moe.KVCache(st["k_pages"], st["v_pages"], n_heads=case["Hq"], inv_freq=st["inv_freq"].numpy(),
                               interleaved=case.get("interleaved", False),
                               k_scale=st["k_scale"].numpy() if e4m3 else None,
                               v_scale=st["v_scale"].numpy() if e4m3 else None, max_batch=max_batch)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        st["x"] = torch.randn(T, H, generator=g, device=DEV).mul_(3).to(KINDS[case["res"]])
        st["o"] = torch.randn(T, H, generator=g, device=DEV).to(KINDS[case["o"]])
        rows = {"none": 0, "row": 1, "full": T}[case["gate"]]
        st["gate"] = torch.rand(rows, H, generator=g, device=DEV).to(KINDS[case["o"]]) if rows else None
        mid = 1.0 - case["offset"]
        st["w_post"] = (torch.randn(H, generator=g, device=DEV) * 0.2 + mid) if case["post"] else None
        st["w_pre"] = torch.randn(H, generator=g, device=DEV) * 0.2 + mid
        st["r"] = torch.empty_like(st["x"])
        st["h"] = torch.empty(T, H, device=DEV, dtype=KINDS[case["h"]])
        if own:
            import quantized_routed_expert_moe_gb300 as moe
            st["norm"] = moe.BlockNorm(H, w_post=st["w_post"], w_pre=st["w_pre"], eps=1e-6, scale=case["scale"],
                                       weight_offset=case["offset"])
        return st
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    rng = random.Random(seed)
    if case["op"] == "attend":
        lens = _lens(case)
        B, width = case["B"], max(1, -(-case["max_len"] // page))
        need = [-(-n // page) for n in lens]
        n_pages = sum(need) + 3
        order = torch.randperm(n_pages, generator=g, device=DEV, dtype=torch.int32)
        table = torch.full((B, width), -1, device=DEV, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        st["table"] = table
        st["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
        # queries a little longer than unit normal: some positions stand out
        st["q"] = (torch.randn(B, Hq, D, generator=g, device=DEV) * 1.5).to(torch.bfloat16)
        st["scale"] = D ** -0.5
        st["out"] = torch.empty(B, Hq, D, device=DEV, dtype=torch.bfloat16)
        st["lse"] = torch.empty(B, Hq, device=DEV, dtype=torch.float32)
        _cache(case, st, n_pages, seed, g, B)
        return st
    T, seqs = case["T"], case["seqs"]
    run_len = T // seqs
    starts = [rng.randrange(max(1, case["far"] - run_len)) for _ in range(seqs)]
    starts[0] = max(0, case["far"] - run_len)
    width = -(-case["far"] // page) + 1 + run_len // page
    pages_each = run_len // page + 2
    n_pages = seqs * pages_each + 1
    order = torch.randperm(n_pages, generator=g, device=DEV, dtype=torch.int32)
    table = torch.zeros(seqs, width, device=DEV, dtype=torch.int32)
    pos, seq = [], []
    for b, s in enumerate(starts):
        first, last = s // page, (s + run_len - 1) // page
        table[b, first:last + 1] = order[b * pages_each:b * pages_each + last - first + 1]
        pos += range(s, s + run_len)
        seq += [b] * run_len
    if T >= 8:
        pos[rng.randrange(T)] = -1  # a padding token
    st["table"] = table
    st["pos"] = torch.tensor(pos, device=DEV, dtype=torch.int32)
    st["seq"] = torch.tensor(seq, device=DEV, dtype=torch.int32)
    # one projection's output: queries, keys and values of a token side by side
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=DEV).to(torch.bfloat16)
    st["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    st["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    st["q_out"] = torch.empty(T, Hq, D, device=DEV, dtype=torch.bfloat16)
    _cache(case, st, n_pages, seed, g, seqs)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rms(x, w, offset):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (w + offset)


def _plain_norm(case, st):
    x, o = st["x"].float(), st["o"].float()
    if st["w_post"] is not None:
        o = _rms(o, st["w_post"], case["offset"])
    if st["gate"] is not None:
        o = o * st["gate"].float()
    r = x + case["scale"] * o
    h = _rms(r, st["w_pre"], case["offset"])
    return {"r": r.to(KINDS[case["res"]]), "h": h.to(KINDS[case["h"]])}


def _rotate(x, cos, sin, rot, interleaved):
    """x [T, heads, D] in 32 bits; cos and sin [T, 1, rot / 2]."""
    y = x.clone()
    if rot:
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        if interleaved:
            y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = ra, rb
    return y


def _to_cache(x, scale, kind):
    if kind == "e4m3":
        return (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return x.to(torch.bfloat16)


def _put(pool, page, slot, x):
    # 8-bit values are placed as the bytes they are
    if pool.dtype == torch.float8_e4m3fn:
        pool, x = pool.view(torch.uint8), x.view(torch.uint8)
    pool[page, :, slot] = x


def _plain_append(case, st):
    pos = st["pos"].long()
    live = pos >= 0
    rot = case["rotary"]
    angle = pos[:, None].double() * st["inv_freq_dev"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotate(st["q"].float(), cos, sin, rot, case["interleaved"])
    k = _rotate(st["k"].float(), cos, sin, rot, case["interleaved"])
    q_out = torch.where(live[:, None, None], q, 0.0).to(torch.bfloat16)
    at = pos[live]
    page = st["table"][st["seq"].long()[live], at // case["page"]].long()
    _put(st["k_pages"], page, at % case["page"], _to_cache(k[live], st["k_scale_dev"], case["cache"]))
    _put(st["v_pages"], page, at % case["page"], _to_cache(st["v"][live].float(), st["v_scale_dev"], case["cache"]))
    return {"q": q_out, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _gather(pool, table, scale):
    """[B, Hkv, width * page, D] in 32 bits."""
    x = pool.view(torch.uint8)[table].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[table]
    x = x.transpose(1, 2).flatten(2, 3).float()
    return x if pool.dtype == torch.bfloat16 else x * scale[:, None, None]


def _plain_attend(case, st):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    table = st["table"].clamp(min=0).long()
    k = _gather(st["k_pages"], table, st["k_scale_dev"])
    q = st["q"].float().view(B, Hkv, Hq // Hkv, D)
    s = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    del k
    if case["softcap"]:
        s = case["softcap"] * torch.tanh(s / case["softcap"])
    j = torch.arange(s.shape[-1], device=s.device)[None, :]
    n = st["lens"][:, None]
    seen = j < n
    if case["window"]:
        seen &= j >= n - case["window"]
    s = torch.where(seen[:, None, None], s, -torch.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -torch.inf, 0.0, m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    v = _gather(st["v_pages"], table, st["v_scale_dev"])
    out = torch.matmul(p, v) / torch.where(l == 0, 1.0, l)
    lse = (m + torch.log(l)).view(B, Hq)
    return {"out": out.view(B, Hq, D).to(torch.bfloat16), "lse": lse}


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "append": _plain_append, "attend": _plain_attend}[op](case, state)
    stream = torch.cuda.current_stream()
    if op == "norm":
        state["norm"].run(state["x"], state["o"], state["r"], state["h"], gate=state["gate"], stream=stream)
        return {"r": state["r"], "h": state["h"]}
    if op == "append":
        state["kv"].append(state["q"], state["k"], state["v"], state["pos"], state["table"], state["q_out"],
                           seq=state["seq"], stream=stream)
        return {"q": state["q_out"], "k_pages": state["k_pages"], "v_pages": state["v_pages"]}
    state["kv"].attend(state["q"], state["table"], state["lens"], state["out"], lse=state["lse"],
                       scale=state["scale"], softcap=case["softcap"], window=case["window"], stream=stream)
    return {"out": state["out"], "lse": state["lse"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["H"]
        gate = {"none": 0, "row": case["H"], "full": n}[case["gate"]]
        b = n * (2 * SIZE[case["res"]] + SIZE[case["o"]] + SIZE[case["h"]]) + gate * SIZE[case["o"]]
        return {"bytes": b + case["H"] * 4 * (2 if case["post"] else 1), "flops": n * 12}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        T = case["T"]
        b = T * ((2 * Hq + 2 * Hkv) * D * 2 + 2 * Hkv * D * SIZE[case["cache"]] + 12)
        return {"bytes": b, "flops": T * (Hq + Hkv) * case["rotary"] * 3}
    seen = [min(n, case["window"]) if case["window"] else n for n in _lens(case)]
    pages = sum(-(-n // case["page"]) for n in seen)
    b = sum(seen) * Hkv * D * 2 * SIZE[case["cache"]] + case["B"] * (Hq * (D * 4 + 4) + 4) + pages * 4
    return {"bytes": b, "flops": 4 * sum(seen) * Hq * D}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits, one sequence and head at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        x, z = st["x"].to(torch.float64), st["o"].to(torch.float64)

        def unit(a):
            return a / torch.sqrt(torch.linalg.vector_norm(a, dim=1, keepdim=True) ** 2 / case["H"] + 1e-6)

        if case["post"]:
            z = unit(z) * (st["w_post"].double() + case["offset"])
        if case["gate"] != "none":
            z = st["gate"].double() * z
        r = torch.add(x, z, alpha=case["scale"])
        return {"r": r, "h": unit(r) * (st["w_pre"].double() + case["offset"])}
    page = case["page"]
    if case["op"] == "append":
        rot, pos, seq = case["rotary"], st["pos"].tolist(), st["seq"].tolist()
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           torch.outer(st["pos"].double(), st["inv_freq_dev"]))[:, None]

        def spun(x):
            x = x.double()
            head, rest = x[..., :rot], x[..., rot:]
            if case["interleaved"]:
                head = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * turn)
                head = head.flatten(-2)
            else:
                z = torch.complex(*head.contiguous().chunk(2, -1)) * turn
                head = torch.cat((z.real, z.imag), -1)
            return torch.cat((head, rest), -1)

        live = [t for t in range(case["T"]) if pos[t] >= 0]
        table = st["table"].cpu()
        pages = torch.tensor([int(table[seq[t], pos[t] // page]) for t in live], device=DEV)
        slots = torch.tensor([pos[t] % page for t in live], device=DEV)
        live = torch.tensor(live, device=DEV)
        got = {"q": torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)}
        got["q"][live] = (spun(st["q"]) if rot else st["q"].double())[live]
        for name in ("k", "v"):
            x = spun(st[name]) if rot and name == "k" else st[name].double()
            if case["cache"] == "e4m3":
                x = (x / st[name + "_scale_dev"].double()[None, :, None]).clamp(-448, 448)
            pool = st[name + "_pages"].to(torch.float32).double()
            pool[pages, :, slots] = x[live]
            got[name + "_pages"] = pool
        return got
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lens(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        at = torch.arange(lo, n, device=DEV)
        pg, sl = st["table"][b, at // page].long(), at % page
        for h in range(Hkv):
            rows = []
            for name in ("k", "v"):
                pool = st[name + "_pages"][:, h]
                if case["cache"] == "e4m3":
                    x = pool.view(torch.uint8)[pg, sl].view(torch.float8_e4m3fn).float().double()
                    rows.append(x * float(st[name + "_scale"][h]))
                else:
                    rows.append(pool[pg, sl].double())
            z = st["q"][b, h * G:(h + 1) * G].double() @ rows[0].T * st["scale"]
            if case["softcap"]:
                z = torch.tanh(z / case["softcap"]) * case["softcap"]
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(z, 1)
            out[b, h * G:(h + 1) * G] = torch.softmax(z, 1) @ rows[1]
    return {"out": out, "lse": lse}
