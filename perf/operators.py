"""Cases of the beam-decoding step on a paged cache, for measurement: the per-head
norm and position rotation of queries and keys (``qk_norm_rope``), the same fused
with the append to the pages (``kv_append_rope`` and its int8/int4 forms), the
selection of the best continuations over beams and vocabulary (``beam_select``)
and the reordering of the cache behind it (``beam_reorder``).

``run`` computes each operator from elementary torch operations, or, where ``own``
is set, calls the library. ``exact`` restates the definitions in 64 bits (numpy).
"""
import numpy as np
import torch

own = False

HEAD_DIM = 128
PAGE = 256
ROPE_BASE = 500000.0  # the base of the rotation frequencies
EPS = 1e-6
CODE_MAX = {"q8": 127, "q4": 7}


# ----------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token, 32 query and 8 KV heads: latency
        {"name": "qk 1 token 32q8kv", "op": "qk", "tokens": 1, "hq": 32, "hkv": 8, "norm": True, "rotary": 128, "interleaved": False},
        # eight prompts' 512-token chunks
        {"name": "qk 4096 tokens 32q8kv", "op": "qk", "tokens": 4096, "hq": 32, "hkv": 8, "norm": True, "rotary": 128, "interleaved": False},
        # an odd number of tokens, half of each head rotated in neighbouring pairs, no norm
        {"name": "qk 1037 tokens 64q8kv half", "op": "qk", "tokens": 1037, "hq": 64, "hkv": 8, "norm": False, "rotary": 64, "interleaved": True},
        # the 64-sequence decode batch: one token each
        {"name": "append decode 64 bf16", "op": "append", "pages": "bf16", "seqs": 64, "new": 1, "ragged": False, "ctx": 1024, "hq": 32, "hkv": 8, "norm": True, "rotary": 128, "interleaved": False},
        # a chunk of 512 new tokens behind 3584 cached ones, eight sequences
        {"name": "append prefill 8x512 bf16", "op": "append", "pages": "bf16", "seqs": 8, "new": 512, "ragged": False, "ctx": 4096, "hq": 32, "hkv": 8, "norm": True, "rotary": 128, "interleaved": False},
        # fresh prompts into int8 pages
        {"name": "append prefill 8x512 int8", "op": "append", "pages": "q8", "seqs": 8, "new": 512, "ragged": False, "ctx": 512, "hq": 32, "hkv": 8, "norm": False, "rotary": 128, "interleaved": False},
        # a mixed batch (nothing, one token, a draft to verify, part of a prompt) into int4 pages
        {"name": "append ragged 24 int4", "op": "append", "pages": "q4", "seqs": 24, "new": 300, "ragged": True, "ctx": 700, "hq": 8, "hkv": 2, "norm": True, "rotary": 64, "interleaved": False},
        # one user's four beams over a small vocabulary: latency
        {"name": "select 1x4 of 32000", "op": "select", "groups": 1, "width": 4, "picks": 4, "vocab": 32000, "dtype": "f32", "ends": False, "first": False},
        # thirteen users' five beams, bf16 logits of an odd vocabulary, twice as many picks as beams, some beams finished
        {"name": "select 13x5 of 50257 bf16", "op": "select", "groups": 13, "width": 5, "picks": 10, "vocab": 50257, "dtype": "bf16", "ends": True, "first": False},
        # thirty-two users' eight beams over the 128256-token vocabulary
        {"name": "select 32x8 of 128256", "op": "select", "groups": 32, "width": 8, "picks": 8, "vocab": 128256, "dtype": "f32", "ends": True, "first": False},
        # one user's four beams on int8 pages
        {"name": "reorder 1x4 int8", "op": "reorder", "pages": "q8", "groups": 1, "width": 4, "ctx": 1000, "hkv": 8},
        # thirty-two users' eight beams, the partial page nearly full
        {"name": "reorder 32x8 bf16", "op": "reorder", "pages": "bf16", "groups": 32, "width": 8, "ctx": 1023, "hkv": 8},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return int(min(hi, max(lo, round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["qk", "append", "select", "reorder"])
    hkv, grp = rng.choice([(1, 8), (2, 4), (3, 5), (4, 2), (4, 1), (8, 4), (8, 8)])
    rope = {"norm": rng.random() < 0.6, "rotary": rng.choice([16, 32, 64, 80, 96, 128, 128, 128]), "interleaved": rng.random() < 0.3}
    if op == "qk":
        return {"op": op, "tokens": _log(rng, 1, 4096 * 40 // max(40, hkv * (grp + 1))), "hq": hkv * grp, "hkv": hkv, **rope}
    if op == "append":
        seqs = _log(rng, 1, 128)
        new = _log(rng, 1, max(1, min(512, 4096 // seqs)))
        return {"op": op, "pages": rng.choice(["bf16", "q8", "q4"]), "seqs": seqs, "new": new, "ragged": rng.random() < 0.5, "ctx": new + rng.randrange(0, 1500),
                "hq": hkv * min(grp, 4), "hkv": hkv, **rope}
    if op == "select":
        width = rng.randrange(1, 17)
        vocab = _log(rng, 500, 200000)
        groups = _log(rng, 1, max(1, min(128, 32000000 // (width * vocab))))
        return {"op": op, "groups": groups, "width": width, "picks": min(32, width * rng.choice([1, 1, 2])), "vocab": vocab, "dtype": rng.choice(["f32", "bf16"]),
                "ends": rng.random() < 0.5, "first": rng.random() < 0.2}
    width = rng.randrange(2, 17)
    return {"op": op, "pages": rng.choice(["bf16", "q8", "q4"]), "groups": _log(rng, 1, max(1, 224 // width)), "width": width, "ctx": rng.randrange(1, 1500), "hkv": hkv}


# ---------------------------------------------------------------------- inputs
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _lens(case):
    """Lengths of one append, from the case alone: new tokens of each sequence and its whole length."""
    rng = np.random.default_rng([case["seqs"], case["new"], case["ctx"]])
    n, new, ctx = case["seqs"], case["new"], case["ctx"]
    q_lens = np.full(n, new, np.int32)
    if case["ragged"]:
        kinds = np.array([0, 1, min(6, new), max(1, new // 3), new], np.int32)
        q_lens = kinds[rng.integers(0, len(kinds), n)]
        q_lens[0] = new
    lo = np.maximum(q_lens, max(new, ctx // 2))
    seq_lens = (lo + rng.integers(0, max(1, ctx - ctx // 2), n) if case["ragged"] or new == 1 else np.full(n, ctx)).astype(np.int32)
    return np.minimum(seq_lens, max(ctx, new)).astype(np.int32), q_lens


def _tables(seq_lens, rng):
    need = (seq_lens + PAGE - 1) // PAGE
    pages = int(need.sum()) + 3
    free = rng.permutation(pages).astype(np.int32)
    table = np.full((len(seq_lens), max(1, int(need.max()))), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = free[at:at + k]
        at += k
    return table, pages


def _pools(gen, dev, kind, pages, hkv):
    """K and V pools as one tensor each of codes and scales (index 0: K, 1: V)."""
    shape = (2, pages, hkv, PAGE)
    if kind == "bf16":
        return {"pages": torch.randn(*shape, HEAD_DIM, generator=gen, device=dev, dtype=torch.float32).to(torch.bfloat16)}
    scales = torch.rand(shape, generator=gen, device=dev) * 0.02 + 0.01
    if kind == "q8":
        return {"codes": torch.randint(-127, 128, (*shape, HEAD_DIM), generator=gen, device=dev, dtype=torch.int8), "scales": scales}
    lo, hi = (torch.randint(1, 16, (*shape, HEAD_DIM // 2), generator=gen, device=dev, dtype=torch.uint8) for _ in range(2))
    return {"codes": lo | (hi << 4), "scales": scales}


def _rope_inputs(case, gen, dev):
    half = case["rotary"] // 2
    # the frequencies as a model's configuration gives them, in 32 bits
    inv = torch.from_numpy((ROPE_BASE ** (-np.arange(half, dtype=np.float64) / half)).astype(np.float32)).to(dev)
    w = [torch.rand(HEAD_DIM, generator=gen, device=dev) + 0.5 for _ in range(2)] if case["norm"] else [None, None]
    return {"inv_freq": inv, "q_weight": w[0], "k_weight": w[1], "rotary": case["rotary"], "interleaved": case["interleaved"]}


def _qkv(case, tokens, gen, dev):
    """Queries, keys and values as the views of one projection's output that a model has."""
    hq, hkv = case["hq"], case["hkv"]
    qkv = torch.randn(tokens, hq + 2 * hkv, HEAD_DIM, generator=gen, device=dev).to(torch.bfloat16)
    return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]


def _inputs(case, seed):
    """The inputs of a case, from its seed alone."""
    dev = _device()
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    s = {"case": case}
    if case["op"] == "qk":
        n = case["tokens"]
        s["q"], s["k"], _ = _qkv(case, n, gen, dev)
        # positions of one long context, and of a batch's sequences behind it
        s["positions"] = put(((np.arange(n) + rng.integers(0, 1 << 20)) % (1 << 20)).astype(np.int32))
        s["rope"] = _rope_inputs(case, gen, dev)
    elif case["op"] == "append":
        seq_lens, q_lens = _lens(case)
        table, pages = _tables(seq_lens, rng)
        total = int(q_lens.sum())
        s["q"], s["k"], s["v"] = _qkv(case, total, gen, dev)
        s |= _pools(gen, dev, case["pages"], pages, case["hkv"])
        s |= {"table": put(table), "seq_lens": put(seq_lens), "q_lens": put(q_lens), "total": total, "max_new": int(q_lens.max()), "num_pages": pages}
        s["rope"] = _rope_inputs(case, gen, dev)
    elif case["op"] == "select":
        b, w, v = case["groups"], case["width"], case["vocab"]
        # a language model's logits: a broad bulk and a few likely tokens in each row
        x = torch.randn(b, w, v, generator=gen, device=dev) * 2.5
        likely = torch.randint(0, v, (b, w, 24), generator=gen, device=dev)
        x.scatter_(2, likely, torch.randn(b, w, 24, generator=gen, device=dev) * 2.0 + 13.0)
        s["logits"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        s["scores"] = -6.0 * torch.rand(b, w, generator=gen, device=dev) - 10.0
        if case["first"]:  # the first step: only beam 0 is in use
            s["scores"] = torch.full_like(s["scores"], -torch.inf)
            s["scores"][:, 0] = 0.0
        s["finished"] = (torch.rand(b, w, generator=gen, device=dev) < 0.15).int() if case["ends"] and not case["first"] else None
        s["eos"] = v // 3 if s["finished"] is not None else -1
    else:
        b, w, t = case["groups"], case["width"], case["ctx"]
        full = t // PAGE
        pages = b * (full + 2 * w) + 3
        free = rng.permutation(pages).astype(np.int32)
        table = np.empty((b, w, full + 2), np.int32)
        table[:, :, :full] = free[:b * full].reshape(b, 1, full)       # the prompt's full pages, shared
        table[:, :, full:] = free[b * full:b * (full + 2 * w)].reshape(b, w, 2)  # each beam's own
        s |= _pools(gen, dev, case["pages"], pages, case["hkv"])
        parents = np.minimum(w - 1, (w * rng.random((b, w)) ** 1.7)).astype(np.int32)
        s |= {"table": put(table.reshape(b * w, -1)), "parents": put(parents), "num_pages": pages,
              "seq_lens": put(np.full(b * w, t, np.int32))}
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    dev = _device()
    op = case["op"]
    if op in ("qk", "append"):
        s["q_out"] = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device=dev)
    if op == "qk":
        s["k_out"] = torch.zeros(s["k"].shape, dtype=torch.bfloat16, device=dev)
    if op in ("append", "reorder") and case["pages"] != "bf16":
        s["values"] = torch.zeros(*s["scales"].shape, HEAD_DIM, dtype=torch.bfloat16, device=dev)  # for the values the codes stand for
        if case["pages"] == "q4":
            byte = torch.arange(256, device=dev)
            s["lut"] = torch.stack([(byte & 15) - 8, (byte >> 4) - 8], 1).to(torch.bfloat16)  # the two values of a byte
    if op == "reorder":
        s["table_out"] = torch.zeros_like(s["table"])
    if own:
        import speculative_decode_gb300 as sa
        s["sa"] = sa
        s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
        if op in ("qk", "append"):
            r = s["rope"]
            s["rope_h"] = sa.Rope(r["inv_freq"], rotary_dim=r["rotary"], interleaved=r["interleaved"], q_weight=r["q_weight"], k_weight=r["k_weight"], eps=EPS)
        if op in ("append", "reorder"):  # the cache as the library takes it: K and V pools (and their scales)
            s["pools"] = tuple(s[n][i] for n in ("pages", "codes", "scales") if n in s for i in range(2))
        if op == "append":
            s["dims"] = sa.dims_for(case["seqs"], case["hq"], case["hkv"], s["num_pages"], s["table"].shape[1], s["total"], s["max_new"])
        if op == "reorder":
            s["dims"] = sa.dims_for(case["groups"] * case["width"], case["hkv"], case["hkv"], s["num_pages"], s["table"].shape[1], case["groups"] * case["width"], 1)
        if op == "select":
            b, w, v, k = case["groups"], case["width"], case["vocab"], case["picks"]
            s["ws"] = torch.zeros(sa.beam_select_workspace_size(b, w, v, k), dtype=torch.uint8, device=dev)
            s["tokens"], s["from"] = (torch.zeros(b, k, dtype=torch.int32, device=dev) for _ in range(2))
            s["scores_out"] = torch.zeros(b, k, device=dev)
            s["finished_out"] = torch.zeros(b, k, dtype=torch.int32, device=dev) if s["finished"] is not None else None
    return s


# ----------------------------------------------------------------- plain forms
def _norm_rope(x, weight, positions, r):
    """Norm of each head and rotation, 32 bits (angles in 64); x [N, H, 128]."""
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight
    rot, half = r["rotary"], r["rotary"] // 2
    angle = positions.double()[:, None] * r["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if r["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _quantise(x, kind):
    top = CODE_MAX[kind]
    amax = x.abs().amax(-1)
    scale = amax / torch.full_like(amax, top)  # a division, not a product with the reciprocal: halves are met exactly
    codes = torch.where(scale[..., None] > 0, (x / scale[..., None]).round().clamp(-top, top), 0.0)
    if kind == "q8":
        return codes.to(torch.int8), scale
    nib = (codes + 8).to(torch.uint8)
    return nib[..., 0::2] | (nib[..., 1::2] << 4), scale


def _page_values(s):
    """The values that the pools stand for."""
    kind = s["case"]["pages"]
    if kind == "bf16":
        return s["pages"]
    if kind == "q8":
        return torch.mul(s["codes"], s["scales"][..., None], out=s["values"])
    return torch.mul(s["lut"][s["codes"].int()].flatten(-2), s["scales"][..., None], out=s["values"])


def _plain_append(s):
    kind, total = s["case"]["pages"], s["total"]
    seq = torch.repeat_interleave(s["q_lens"], output_size=total)
    first = s["q_lens"].cumsum(0) - s["q_lens"]
    pos = (s["seq_lens"] - s["q_lens"] - first)[seq] + torch.arange(total, device=seq.device)
    s["q_out"].copy_(_norm_rope(s["q"], s["rope"]["q_weight"], pos, s["rope"]))
    page, slot = s["table"][seq, pos // PAGE].long(), pos % PAGE
    both = torch.stack([_norm_rope(s["k"], s["rope"]["k_weight"], pos, s["rope"]), s["v"].float()])
    if kind == "bf16":
        s["pages"][:, page, :, slot] = both.to(torch.bfloat16).transpose(0, 1)
    else:
        codes, scales = _quantise(both, kind)
        s["codes"][:, page, :, slot] = codes.transpose(0, 1)
        s["scales"][:, page, :, slot] = scales.transpose(0, 1)
    return {"q": s["q_out"], "pages": _page_values(s)}


def _plain_select(s):
    case = s["case"]
    b, w, v, k = case["groups"], case["width"], case["vocab"], case["picks"]
    x = s["logits"].float()
    x = torch.where(x.isnan(), -torch.inf, x).clamp(max=torch.finfo(torch.float32).max)
    wide = x.double()
    top = wide.amax(-1, keepdim=True)
    lse = (wide - top).exp().sum(-1, keepdim=True).log() + top
    best, token = x.sort(dim=-1, descending=True, stable=True)
    best, token = best[..., :k].double(), token[..., :k]
    value = s["scores"].double()[..., None] + (best - lse)
    value = torch.where(value.isnan(), -torch.inf, value)
    if s["finished"] is not None:
        # a finished beam goes on with its end token alone, at its own score
        done = s["finished"][..., None] != 0
        rank = torch.arange(best.shape[-1], device=x.device)
        rest = torch.where(rank == 0, s["eos"], torch.where(rank - 1 < s["eos"], rank - 1, rank))
        token = torch.where(done, rest, token)
        value = torch.where(done, torch.where(rank == 0, s["scores"].double()[..., None], -torch.inf), value)
    value, at = value.flatten(1).sort(dim=-1, descending=True, stable=True)
    value, at = value[:, :k], at[:, :k]
    parents = at // best.shape[-1]
    out = {"tokens": token.flatten(1).gather(1, at).int(), "parents": parents.int(), "scores": value.float()}
    if s["finished"] is not None:
        out["finished"] = ((s["finished"].gather(1, parents) != 0) | (out["tokens"] == s["eos"])).int()
    return out


def _plain_reorder(s):
    case = s["case"]
    b, w, t = case["groups"], case["width"], case["ctx"]
    full, rows = t // PAGE, t % PAGE
    dev = s["table"].device
    p = s["parents"].long()
    beam = torch.arange(w, device=dev)
    same = p[:, :, None] == p[:, None, :]
    heir = ~(same & (beam[None, :] < beam[:, None])).any(-1)          # no lower child of the same parent
    childless = ~(p[:, :, None] == beam).any(1)
    # the k-th other child takes the k-th childless beam's pages
    order = torch.where(childless, beam, w + beam).sort(-1)[0] % w
    rank = (~heir).long().cumsum(-1) - 1
    donor = torch.where(heir, p, order.gather(1, rank.clamp(min=0)))
    group = torch.arange(b, device=dev)[:, None]
    table = s["table"].view(b, w, -1)
    new = torch.cat([table[group, p][..., :full], table[group, donor][..., full:]], -1)
    s["table_out"].copy_(new.view(b * w, -1))
    if rows:
        src, dst = table[group, p][..., full].flatten().long(), new[..., full].flatten().long()
        for name in ("pages", "codes", "scales"):
            if name in s:
                # a child that kept its page copies it onto itself
                s[name][:, dst, :, :rows] = s[name][:, src, :, :rows]
    return {"table": s["table_out"], "pages": _page_values(s)}


# ------------------------------------------------------------------------- run
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "qk":
            r = s["rope"]
            s["q_out"].copy_(_norm_rope(s["q"], r["q_weight"], s["positions"], r))
            s["k_out"].copy_(_norm_rope(s["k"], r["k_weight"], s["positions"], r))
            return {"q": s["q_out"], "k": s["k_out"]}
        return {"append": _plain_append, "select": _plain_select, "reorder": _plain_reorder}[op](s)
    sa = s["sa"]
    if op == "qk":
        sa.qk_norm_rope(s["rope_h"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "select":
        sa.beam_select(s["logits"], s["scores"], s["tokens"], s["from"], s["scores_out"], s["ws"], finished=s["finished"], finished_out=s["finished_out"], eos_token=s["eos"])
        out = {"tokens": s["tokens"], "parents": s["from"], "scores": s["scores_out"]}
        return out if s["finished"] is None else {**out, "finished": s["finished_out"]}
    if op == "append":
        call = {"bf16": sa.kv_append_rope, "q8": sa.kv_append_rope_q8, "q4": sa.kv_append_rope_q4}[case["pages"]]
        call(s["dims"], s["rope_h"], s["q"], s["k"], s["v"], s["q_out"], *s["pools"], s["table"], s["seq_lens"], s["q_lens"], err_flag=s["err"])
        return {"q": s["q_out"], "pages": _page_values(s)}
    call = {"bf16": sa.beam_reorder, "q8": sa.beam_reorder_q8, "q4": sa.beam_reorder_q4}[case["pages"]]
    call(s["dims"], case["width"], s["parents"], s["table"], s["seq_lens"], s["table_out"], *s["pools"], err_flag=s["err"])
    return {"table": s["table_out"], "pages": _page_values(s)}


# ------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    row = {"bf16": 2 * HEAD_DIM, "q8": HEAD_DIM + 4, "q4": HEAD_DIM // 2 + 4}.get(case.get("pages"))
    if op == "qk":
        heads = case["hq"] + case["hkv"]
        n = case["tokens"]
        return {"bytes": n * (heads * 4 * HEAD_DIM + 4), "flops": 10 * n * heads * HEAD_DIM}
    if op == "append":
        seq_lens, q_lens = _lens(case)
        n = int(q_lens.sum())
        hq, hkv = case["hq"], case["hkv"]
        return {"bytes": n * (hq * 4 * HEAD_DIM + hkv * (4 * HEAD_DIM + 2 * row)) + 16 * case["seqs"], "flops": 10 * n * (hq + 2 * hkv) * HEAD_DIM}
    if op == "select":
        n = case["groups"] * case["width"] * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + case["groups"] * (case["width"] * 8 + case["picks"] * 16), "flops": 4 * n}
    # about a third of the beams are copied; the tables are read and written
    b, w, t = case["groups"], case["width"], case["ctx"]
    parents = _inputs_parents(case, 0)
    extra = sum(w - len(set(g)) for g in parents)
    return {"bytes": extra * (t % PAGE) * case["hkv"] * row * 2 * 2 + b * w * (t // PAGE + 2) * 8 + b * w * 4, "flops": 0}


def _inputs_parents(case, seed):
    """Parents of the distribution that the inputs have (for counting)."""
    rng = np.random.default_rng(seed)
    w = case["width"]
    return np.minimum(w - 1, (w * rng.random((case["groups"], w)) ** 1.7)).astype(np.int32).tolist()


# ----------------------------------------------------------------------- exact
def _np(t):
    return t.double().cpu().numpy()


def _exact_rows(x, weight, pos, r):
    """Norm and rotation by complex multiplication, 64 bits."""
    y = _np(x)
    if weight is not None:
        y = y / np.sqrt(np.einsum("nhd,nhd->nh", y, y) / HEAD_DIM + EPS)[..., None] * _np(weight)
    rot = r["rotary"]
    turn = np.exp(1j * np.outer(pos.astype(np.float64), _np(r["inv_freq"])))[:, None]
    i = np.arange(0, rot, 2) if r["interleaved"] else np.arange(rot // 2)
    j = i + (1 if r["interleaved"] else rot // 2)
    z = (y[..., i] + 1j * y[..., j]) * turn
    y[..., i], y[..., j] = z.real, z.imag
    return y


def exact(case, seed):
    op = case["op"]
    if op == "reorder":  # moves rows, computes no numbers
        return None
    s = _inputs(case, seed)
    if op == "qk":
        pos = s["positions"].cpu().numpy()
        return {"q": _exact_rows(s["q"], s["rope"]["q_weight"], pos, s["rope"]), "k": _exact_rows(s["k"], s["rope"]["k_weight"], pos, s["rope"])}
    if op == "append":
        seq_lens, q_lens, table = (s[n].cpu().numpy() for n in ("seq_lens", "q_lens", "table"))
        kind = case["pages"]
        pos = np.concatenate([np.arange(t - n, t) for t, n in zip(seq_lens, q_lens)])
        seq = np.concatenate([np.full(n, b) for b, n in enumerate(q_lens)])
        if kind == "bf16":
            pages = _np(s["pages"])
        elif kind == "q8":
            pages = _np(s["codes"]) * _np(s["scales"])[..., None]
        else:
            c = s["codes"].cpu().numpy()
            pages = (np.stack([c % 16, c // 16], -1).reshape(*c.shape[:-1], HEAD_DIM).astype(np.float64) - 8) * _np(s["scales"])[..., None]
        rows = np.stack([_exact_rows(s["k"], s["rope"]["k_weight"], pos, s["rope"]), _np(s["v"])])
        if kind != "bf16":
            # the pages' format defines scale and code by two binary32 divisions of the row
            row32 = rows.astype(np.float32)
            step = np.abs(row32).max(-1, keepdims=True) / np.float32(CODE_MAX[kind])
            rows = np.rint(np.divide(row32, step, out=np.zeros_like(row32), where=step > 0)).astype(np.float64) * step
        page = table[seq, pos // PAGE]
        for side in range(2):
            pages[side][page, :, pos % PAGE] = rows[side]
        return {"q": _exact_rows(s["q"], s["rope"]["q_weight"], pos, s["rope"]), "pages": pages}
    w, k, v = case["width"], case["picks"], case["vocab"]
    logits, scores = s["logits"].float().cpu().numpy(), _np(s["scores"])
    done = None if s["finished"] is None else s["finished"].cpu().numpy()
    tokens, parents, values = [], [], []
    for g in range(case["groups"]):
        heap = []
        for i in range(w):
            x = logits[g, i]
            if done is not None and done[g, i]:
                others = [t for t in range(min(v, k + 1)) if t != s["eos"]][:k - 1]
                heap += [(-scores[g, i], i, 0, s["eos"])] + [(np.inf, i, 1 + n, t) for n, t in enumerate(others)]
                continue
            wide = x.astype(np.float64)
            lse = np.log(np.exp(wide - wide.max()).sum()) + wide.max()
            cut = np.partition(x, v - k)[v - k] if k < v else x.min()
            near = np.flatnonzero(x >= cut)
            near = near[np.lexsort((near, -wide[near]))][:k]
            heap += [(-(scores[g, i] + (wide[t] - lse)), i, n, t) for n, t in enumerate(near)]
        heap = sorted(heap)[:k]
        tokens.append([h[3] for h in heap])
        parents.append([h[1] for h in heap])
        values.append([-h[0] for h in heap])
    out = {"tokens": np.array(tokens, np.int32), "parents": np.array(parents, np.int32), "scores": np.array(values)}
    if done is not None:
        out["finished"] = np.array([[int(bool(done[g, p]) or t == s["eos"]) for t, p in zip(tokens[g], parents[g])] for g in range(case["groups"])], np.int32)
    return out
