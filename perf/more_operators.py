"""The operators that take a decoder layer through a chunk of a prompt, as measured cases.

Beside the norms, the cache append and the attention of single tokens, such a pass needs

- ``chunk``   attention of a chunk of new tokens per sequence over the paged cache, each
              token over what stands before it and itself (sequences of different
              lengths packed behind one another);
- ``norm``    the append with the norms of every head's queries and keys in the same pass,
              before the rotation by the position;
- ``linear``  y = act(x W^T + bias) + residual: the projections around the attention.

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

def _chunk(B, new, Hq, Hkv, D, page, far, lens="ragged", cache="bf16", window=0, softcap=0.0, layout="hnd"):
    return dict(op="chunk", B=B, new=new, Hq=Hq, Hkv=Hkv, D=D, page=page, far=far, lens=lens, cache=cache,
                window=window, softcap=softcap, layout=layout)


def _norm(T, seqs, Hq, Hkv, D, page, far, cache="bf16", rotary=None, interleaved=False, layout="hnd", offset=0.0):
    return dict(op="norm", T=T, seqs=seqs, Hq=Hq, Hkv=Hkv, D=D, page=page, far=far, cache=cache,
                rotary=D if rotary is None else rotary, interleaved=interleaved, layout=layout, offset=offset)


def _linear(T, K, N, out="bf16", act="none", bias=False, residual=False):
    return dict(op="linear", T=T, K=K, N=N, out=out, act=act, bias=bias, residual=residual)


def listed():
    return [
        # a short first prompt on the 512-wide layer (8 heads of 64): pure latency
        dict(_chunk(1, 17, 8, 2, 64, 16, 17, "equal"), name="chunk_first_tokens"),
        # one prefill chunk of 128 tokens far into a long document (48 heads of 128): the split over the length
        dict(_chunk(1, 128, 48, 8, 128, 64, 32768, "equal"), name="chunk_far"),
        # a whole prompt at once, nothing cached before it
        dict(_chunk(1, 8192, 48, 8, 128, 64, 8192, "equal"), name="chunk_prompt"),
        # a few drafted tokens of each of 64 conversations to be verified, small pages
        dict(_chunk(64, 4, 48, 8, 128, 16, 16384), name="chunk_drafts"),
        # a serving batch of chunks of different lengths over an 8-bit cache, 16 queries to a key-value head
        dict(_chunk(32, 128, 64, 4, 128, 64, 9001, cache="e4m3"), name="chunk_batch_8bit"),
        # sliding-window layers with capped logits and wide heads, tokens outermost in a page
        dict(_chunk(8, 509, 16, 8, 256, 32, 4500, window=1024, softcap=50.0, layout="nhd"), name="chunk_window_cap"),
        # queries, keys and values of one decode token on the 512-wide layer
        dict(_linear(1, 512, 768, bias=True), name="linear_one_small"),
        # the same on the 6144-wide layer, 48 + 2 * 8 heads of 128
        dict(_linear(1, 6144, 8192), name="linear_one"),
        # the output projection of one prefill chunk onto the fp32 residual stream
        dict(_linear(128, 6144, 6144, out="f32", residual=True), name="linear_chunk"),
        # a long prompt's projection with its activation, on the 2816-wide layer, 16 + 2 * 8 heads of 256
        dict(_linear(8191, 2816, 8192, act="gelu_tanh", bias=True), name="linear_prompt"),
        # one decode token, norms of the heads before the rotation
        dict(_norm(1, 1, 48, 8, 128, 64, 5000), name="norm_one"),
        # chunks of many sequences into an 8-bit cache
        dict(_norm(8192, 64, 48, 8, 128, 64, 60000, cache="e4m3"), name="norm_many_chunks_8bit"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Sizes over the range the listed cases span, odd ones among them."""
    op = rng.choice(("chunk", "chunk", "norm", "linear"))
    if op == "linear":
        T, K, N = _log(rng, 1, 8191), 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 1024)
        while T * K * N > 8191 * 2816 * 8192:
            T = max(1, T // 2)
        return _linear(T, K, N, rng.choice(("bf16", "f32")), rng.choice(("none", "none", "silu", "gelu_tanh", "sigmoid")),
                       rng.random() < 0.5, rng.random() < 0.5)
    D = rng.choice((64, 128, 256))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    G = rng.choice((1, 2, 4, 5, 6, 8, 12, 16))
    page = rng.choice((16, 32, 48, 64, 128))
    cache = rng.choice(("bf16", "bf16", "e4m3"))
    layout = rng.choice(("hnd", "nhd"))
    if op == "norm":
        seqs = _log(rng, 1, 64)
        T = seqs * _log(rng, 1, 110)
        G = min(G, max(1, 40 * 128 // (Hkv * D)))
        return _norm(T, seqs, Hkv * G, Hkv, D, page, _log(rng, 200, 1000000), cache,
                     rng.choice((D, D, D // 2, 0)), rng.random() < 0.4, layout, rng.choice((0.0, 1.0)))
    B = _log(rng, 1, 64)
    lens = rng.choice(("ragged", "equal"))
    new = _log(rng, 1, max(1, 8192 // B))
    far = max(new, _log(rng, 1, 32768))
    window, softcap = rng.choice((0, 0, 0, _log(rng, 1, 4096))), rng.choice((0.0, 0.0, 30.0))
    # no more scores, cached values or products than the largest listed case has
    while True:
        case = _chunk(B, new, Hkv * G, Hkv, D, page, far, lens, cache, window, softcap, layout)
        if (B * new * Hkv * G * far <= 8192 * 48 * 8192 and B * Hkv * D * far <= 64 * 16384 * 8 * 128
                and work(case)["flops"] <= 4 * 48 * 128 * 8192 * 4096):
            return case
        far = max(1, far // 2)
        new = min(new, far)


def _sizes(case):
    """New and cached tokens (the new ones among them) of every sequence: a property of the
    case, so that its work is known."""
    B, new, far = case["B"], case["new"], case["far"]
    if case["lens"] == "equal":
        return [new] * B, [far] * B
    rng = random.Random(B * 1000003 + far)
    chunks = [_log(rng, max(1, new // 16), new) for _ in range(B)]
    chunks[rng.randrange(B)] = new
    lens = [max(n, _log(rng, max(1, far // 16), far)) for n in chunks]
    lens[rng.randrange(B)] = far
    if B >= 8:
        chunks[rng.randrange(1, B)] = 0  # nothing new in this slot
    return chunks, lens


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pool(case, n_pages, g, size):
    """A page pool as [n_pages, Hkv, page, D], its memory in the case's order."""
    Hkv, page, D = case["Hkv"], case["page"], case["D"]
    shape = (n_pages, Hkv, page, D) if case["layout"] == "hnd" else (n_pages, page, Hkv, D)
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    if case["cache"] == "e4m3":
        x = (x * (448 / 5)).clamp_(-448, 448).to(torch.float8_e4m3fn)
    elif size != 1.0:
        x *= size
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


def _prepare_linear(case, st, g):
    T, K, N = case["T"], case["K"], case["N"]
    st["x"] = torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16)
    st["w"] = (torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16)
    st["bias"] = torch.randn(N, generator=g, device=DEV) * 0.3 if case["bias"] else None
    st["residual"] = torch.randn(T, N, generator=g, device=DEV).mul_(2).to(KINDS[case["out"]]) if case["residual"] else None
    st["y"] = torch.empty(T, N, device=DEV, dtype=KINDS[case["out"]])
    if own:
        import quantized_routed_expert_moe_gb300 as moe
        st["linear"] = moe.Linear(st["w"], bias=st["bias"], activation=case["act"])


def _prepare_chunk(case, st, seed, g):
    Hq, D, page, B = case["Hq"], case["D"], case["page"], case["B"]
    chunks, lens = _sizes(case)
    T, width = sum(chunks), max(1, -(-max(lens) // page))
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV, dtype=torch.int32)
    table = torch.full((B, width), -1, device=DEV, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [sum(chunks[:b]) for b in range(B + 1)]
    st["table"] = table
    st["lens"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    st["starts"] = torch.tensor(starts, device=DEV, dtype=torch.int32)
    st["seq"] = torch.tensor([b for b, n in enumerate(chunks) for _ in range(n)], device=DEV)
    st["at"] = torch.tensor([i for n in chunks for i in range(n)], device=DEV)
    # queries a little longer than unit normal: some positions stand out
    st["q"] = (torch.randn(T, Hq, D, generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    st["scale"] = D ** -0.5
    st["out"] = torch.empty(T, Hq, D, device=DEV, dtype=torch.bfloat16)
    st["lse"] = torch.empty(T, Hq, device=DEV, dtype=torch.float32)
    _cache(case, st, n_pages, seed, g, B)


def _prepare_norm(case, st, seed, g):
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    T, seqs = case["T"], case["seqs"]
    rng = random.Random(seed)
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
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=DEV).mul_(2).to(torch.bfloat16)
    st["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    st["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    st["q_norm"] = torch.randn(D, generator=g, device=DEV) * 0.2 + 1 - case["offset"]
    st["k_norm"] = torch.randn(D, generator=g, device=DEV) * 0.2 + 1 - case["offset"]
    st["q_out"] = torch.empty(T, Hq, D, device=DEV, dtype=torch.bfloat16)
    _cache(case, st, n_pages, seed, g, seqs)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "linear":
        _prepare_linear(case, st, g)
    elif case["op"] == "chunk":
        _prepare_chunk(case, st, seed, g)
    else:
        _prepare_norm(case, st, seed, g)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return 1 / (1 + torch.exp(-z)) if act == "sigmoid" else z


def _plain_linear(case, st):
    z = torch.matmul(st["x"].float(), st["w"].float().T)
    if case["bias"]:
        z = z + st["bias"]
    z = _act(z, case["act"])
    if case["residual"]:
        z = z + st["residual"].float()
    return {"y": z.to(KINDS[case["out"]])}


def _rms(x, w, offset):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (w + offset)


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


def _plain_norm(case, st):
    pos = st["pos"].long()
    live = pos >= 0
    rot = case["rotary"]
    angle = pos[:, None].double() * st["inv_freq_dev"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotate(_rms(st["q"].float(), st["q_norm"], case["offset"]), cos, sin, rot, case["interleaved"])
    k = _rotate(_rms(st["k"].float(), st["k_norm"], case["offset"]), cos, sin, rot, case["interleaved"])
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


def _plain_chunk(case, st):
    B, Hq, Hkv, D, new = case["B"], case["Hq"], case["Hkv"], case["D"], case["new"]
    G = Hq // Hkv
    table = st["table"].clamp(min=0).long()
    first, count = st["starts"][:-1].long(), (st["starts"][1:] - st["starts"][:-1]).long()
    i = torch.arange(new, device=DEV)
    rows = (first[:, None] + i).clamp(max=st["q"].shape[0] - 1)
    # [B, Hkv, G * new, D]: the chunks side by side, as long as the longest
    q = st["q"].float()[rows].view(B, new, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * new, D)
    k = _gather(st["k_pages"], table, st["k_scale_dev"])
    s = torch.matmul(q, k.transpose(2, 3)).mul_(st["scale"])
    del k
    if case["softcap"]:
        s = torch.tanh(s / case["softcap"]) * case["softcap"]
    j = torch.arange(s.shape[-1], device=DEV)
    pos = (st["lens"].long() - count)[:, None] + i
    seen = j <= pos[:, :, None]
    if case["window"]:
        seen &= j > pos[:, :, None] - case["window"]
    s = s.view(B, Hkv, G, new, -1).masked_fill_(~seen[:, None, None], -torch.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -torch.inf, 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    v = _gather(st["v_pages"], table, st["v_scale_dev"])
    out = torch.matmul(p.view(B, Hkv, G * new, -1), v).view(B, Hkv, G, new, D)
    out = (out / torch.where(total == 0, 1.0, total)).permute(0, 3, 1, 2, 4).reshape(B, new, Hq, D)
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(B, new, Hq)
    at = st["seq"], st["at"]
    return {"out": out[at].to(torch.bfloat16), "lse": lse[at]}


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "linear": _plain_linear, "chunk": _plain_chunk}[op](case, state)
    stream = torch.cuda.current_stream()
    if op == "linear":
        state["linear"].run(state["x"], state["y"], residual=state["residual"], stream=stream)
        return {"y": state["y"]}
    if op == "norm":
        state["kv"].append(state["q"], state["k"], state["v"], state["pos"], state["table"], state["q_out"],
                           seq=state["seq"], q_norm=state["q_norm"], k_norm=state["k_norm"], norm_eps=1e-6,
                           norm_offset=case["offset"], stream=stream)
        return {"q": state["q_out"], "k_pages": state["k_pages"], "v_pages": state["v_pages"]}
    state["kv"].attend_chunk(state["q"], state["starts"], state["table"], state["lens"], state["out"], lse=state["lse"],
                             scale=state["scale"], softcap=case["softcap"], window=case["window"], stream=stream)
    return {"out": state["out"], "lse": state["lse"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        b = (T + N) * K * 2 + T * N * SIZE[case["out"]] * (2 if case["residual"] else 1) + (N * 4 if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * T * K * N}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "norm":
        T = case["T"]
        b = T * ((2 * Hq + 2 * Hkv) * D * 2 + 2 * Hkv * D * SIZE[case["cache"]] + 12) + 2 * D * 4
        return {"bytes": b, "flops": T * (Hq + Hkv) * (case["rotary"] * 3 + D * 4)}
    chunks, lens = _sizes(case)
    w = case["window"] or max(lens)
    cached = pages = seen = 0
    for n, total in zip(chunks, lens):
        if n:
            lo = max(0, total - n + 1 - w)
            cached += total - lo
            pages += -(-total // case["page"]) - lo // case["page"]
            short = min(max(w - (total - n) - 1, 0), n)  # tokens that see all before them, fewer than the window
            seen += short * (total - n) + short * (short + 1) // 2 + (n - short) * w
    T = sum(chunks)
    b = cached * Hkv * D * 2 * SIZE[case["cache"]] + T * Hq * (D * 4 + 4) + case["B"] * 8 + pages * 4
    return {"bytes": b, "flops": 4 * seen * Hq * D}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits, one sequence and head at a time
# ---------------------------------------------------------------------------

def _exact_linear(case, st):
    z = torch.nn.functional.linear(st["x"].double(), st["w"].double(), st["bias"].double() if case["bias"] else None)
    if case["act"] == "silu":
        z = z * torch.sigmoid(z)
    elif case["act"] == "gelu_tanh":
        z = torch.nn.functional.gelu(z, approximate="tanh")
    elif case["act"] == "sigmoid":
        z = torch.sigmoid(z)
    return {"y": z + st["residual"].double() if case["residual"] else z}


def _exact_norm(case, st):
    page, rot, pos, seq = case["page"], case["rotary"], st["pos"].tolist(), st["seq"].tolist()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.outer(st["pos"].double(), st["inv_freq_dev"]))[:, None]

    def spun(x, w):
        x = x.double()
        x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / case["D"] + 1e-6)
        x = x * (w.double() + case["offset"])
        head, rest = x[..., :rot], x[..., rot:]
        if rot and case["interleaved"]:
            head = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
        elif rot:
            z = torch.complex(*head.contiguous().chunk(2, -1)) * turn
            head = torch.cat((z.real, z.imag), -1)
        return torch.cat((head, rest), -1)

    live = [t for t in range(case["T"]) if pos[t] >= 0]
    table = st["table"].cpu()
    pages = torch.tensor([int(table[seq[t], pos[t] // page]) for t in live], device=DEV)
    slots = torch.tensor([pos[t] % page for t in live], device=DEV)
    live = torch.tensor(live, device=DEV)
    got = {"q": torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)}
    got["q"][live] = spun(st["q"], st["q_norm"])[live]
    for name in ("k", "v"):
        x = spun(st["k"], st["k_norm"]) if name == "k" else st["v"].double()
        if case["cache"] == "e4m3":
            x = (x / st[name + "_scale_dev"].double()[None, :, None]).clamp(-448, 448)
        pool = st[name + "_pages"].to(torch.float32).double()
        pool[pages, :, slots] = x[live]
        got[name + "_pages"] = pool
    return got


def _exact_chunk(case, st):
    Hq, Hkv, D, page, w = case["Hq"], case["Hkv"], case["D"], case["page"], case["window"]
    G = Hq // Hkv
    T = st["q"].shape[0]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    t0 = 0
    for b, (n, total) in enumerate(zip(*_sizes(case))):
        # positions [lo, total) of the cache, of which token i sees those up to its own
        lo = max(0, total - n + 1 - w) if w else 0
        j = torch.arange(lo, total, device=DEV)
        own_pos = torch.arange(total - n, total, device=DEV)[:, None]
        hidden = (j > own_pos) | (j <= own_pos - w) if w else j > own_pos
        pg, sl = st["table"][b, j // page].long(), j % page
        for h in range(Hkv if n else 0):
            rows = []
            for name in ("k", "v"):
                pool = st[name + "_pages"][:, h]
                if case["cache"] == "e4m3":
                    x = pool.view(torch.uint8)[pg, sl].view(torch.float8_e4m3fn).float().double()
                    rows.append(x * float(st[name + "_scale"][h]))
                else:
                    rows.append(pool[pg, sl].double())
            for i in range(h * G, (h + 1) * G):
                z = st["q"][t0:t0 + n, i].double() @ rows[0].T * st["scale"]
                if case["softcap"]:
                    z = torch.tanh(z / case["softcap"]) * case["softcap"]
                z[hidden] = -math.inf
                lse[t0:t0 + n, i] = torch.logsumexp(z, 1)
                out[t0:t0 + n, i] = torch.softmax(z, 1) @ rows[1]
        t0 += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    return {"linear": _exact_linear, "norm": _exact_norm, "chunk": _exact_chunk}[case["op"]](case, st)
