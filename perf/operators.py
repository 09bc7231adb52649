"""What a serving step does around the projections, as operators: keys and values appended to
a paged cache held in 4 bits, attention over that cache, and the choice of the next token.

Each case names one operator and its sizes.  ``run`` computes it in elementary torch
operations, or, with ``own`` set, through this repository's entry points:

  append     K is rotated to its position, each (token, head) row of K and of V is held as 4-bit
             codes c with a scale s and an offset z, x ~ s c + z, and the rows are read back
  attention  softmax(scale q K^T) V over the pages of each sequence, causal, for one new token
             or a run of them; q is rotated on the way
  sample     temperature, top-k, top-p and min-p, and a token drawn with a given uniform number

A row x of the cache, in exact arithmetic: z is the largest bf16 number <= min x, s the bf16
number next to (max x - z) / 15 (ties to even), c = (x - z) / s rounded to a whole number (ties
to even) and kept within 0..15, 0 where s is 0.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
THETA = 500000.0


# ------------------------------------------------------------------ cases --
def listed():
    def append(name, batch, new, past, kv, hd, page, dtype, rope=True):
        return {"name": name, "op": "append", "batch": batch, "new": new, "past": past, "kv": kv, "hd": hd,
                "page": page, "dtype": dtype, "rope": rope}

    def attention(name, batch, new, past, kv, group, hd, page, dtype, rope=True):
        return {"name": name, "op": "attention", "batch": batch, "new": new, "past": past, "kv": kv,
                "group": group, "hd": hd, "page": page, "dtype": dtype, "rope": rope}

    def sample(name, batch, vocab, dtype, top_k, top_p, min_p, masked):
        return {"name": name, "op": "sample", "batch": batch, "vocab": vocab, "dtype": dtype, "top_k": top_k,
                "top_p": top_p, "min_p": min_p, "masked": masked}

    return [
        # one new token of one sequence of the 1B decoder, deep in its context: the smallest call
        append("append_b1", 1, 1, 600, 8, 64, 64, "bf16"),
        # the largest decode batch of the 1B decoder, sequences of many lengths
        append("append_b48", 48, 1, 623, 8, 64, 64, "bf16"),
        # 32 prompts of about 496 tokens at once, no two of the same length
        append("append_prompts", 32, 496, 0, 8, 64, 64, "bf16"),
        # one step of one conversation: little to read, so latency counts
        attention("attend_b1", 1, 1, 623, 8, 4, 64, 64, "bf16"),
        # the 1B decoder's largest batch with the fp32 activations that its GEMV step keeps, rotated already
        attention("attend_b48", 48, 1, 623, 8, 4, 64, 64, "fp32", False),
        # long conversations served together: the cache is what a step reads
        attention("attend_b32_long", 32, 1, 8191, 8, 4, 64, 64, "bf16"),
        # one very long document, heads of 128 in groups of 8: the long axis has to be split
        attention("attend_b1_document", 1, 1, 131071, 8, 8, 128, 64, "fp16"),
        # the next piece of four prompts that are read in pieces
        attention("attend_pieces", 4, 512, 4096, 8, 4, 64, 64, "bf16"),
        # the codebook head's vocabulary, plain temperature: the smallest draw
        sample("sample_codebook", 32, 2048, "fp32", False, False, False, False),
        # one sequence of the 1B decoder, the usual top-p
        sample("sample_b1", 1, 128256, "fp32", False, True, False, False),
        # the 1B decoder's largest batch, every request with settings of its own
        sample("sample_b48", 48, 128256, "fp32", True, True, True, False),
        # a large cohort of constrained requests: most tokens are masked in half of the rows
        sample("sample_b128_masked", 128, 128256, "fp32", True, True, True, True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "sample"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "sample":
        vocab = _log_uniform(rng, 257, 160000)
        batch = _log_uniform(rng, 1, min(128, 16000000 // vocab))
        return {"op": op, "batch": batch, "vocab": vocab, "dtype": dtype, "top_k": rng.random() < 0.5,
                "top_p": rng.random() < 0.6, "min_p": rng.random() < 0.4, "masked": rng.random() < 0.3}
    c = {"op": op, "kv": rng.choice([1, 2, 3, 4, 8]), "hd": rng.choice([64, 64, 128]),
         "page": rng.choice([16, 32, 48, 64, 64, 128]), "dtype": dtype, "rope": rng.random() < 0.7}
    if op == "append":
        c["batch"] = _log_uniform(rng, 1, 64)
        c["new"] = 1 if rng.random() < 0.4 else _log_uniform(rng, 1, 7000 // c["batch"])
        c["past"] = rng.choice([0, _log_uniform(rng, 1, 4000)])
        return c
    c["group"] = rng.choice([1, 2, 3, 4, 4, 7, 8])
    if rng.random() < 0.6:  # single tokens
        c["batch"] = _log_uniform(rng, 1, 64)
        c["new"] = 1
        c["past"] = _log_uniform(rng, 1, 120000 // c["batch"])
    else:  # runs of them
        c["new"] = _log_uniform(rng, 2, 400)
        c["past"] = rng.choice([0, _log_uniform(rng, 1, 3000)])
        one = c["new"] * (c["past"] + c["new"]) * c["kv"] * c["group"] * c["hd"]
        c["batch"] = _log_uniform(rng, 1, max(1, min(6, 10 ** 10 // one)))
    return c


def _lengths(case):
    """Tokens held and tokens new of each sequence: spread below the case's sizes, the first one full."""
    b = np.arange(case["batch"])
    past = case["past"] - (b * 7919 % 101) * case["past"] // 202
    new = np.maximum(1, case["new"] - (b * 104729 % 89) * case["new"] // 178)
    return past, new


def _blocks(case):
    return -(-(case["past"] + case["new"]) // case["page"])


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "sample":
        n = case["batch"] * case["vocab"]
        return {"bytes": n * size + case["batch"] * 32, "flops": 4 * n}
    past, new = _lengths(case)
    kv, hd = case["kv"], case["hd"]
    row = hd // 2 + 4  # bytes of a row in the cache: its codes, its scale and offset
    rows = int(new.sum()) * kv
    if case["op"] == "append":  # the rows come in, are held, and go out again
        return {"bytes": rows * 2 * (2 * hd * size + row), "flops": rows * hd * (11 if case["rope"] else 8)}
    heads = kv * case["group"]
    seen = int((new * past + new * (new + 1) // 2).sum())  # (query, key) pairs of a head
    return {"bytes": int((past + new).sum()) * kv * 2 * row + int(new.sum()) * heads * 2 * hd * size,
            "flops": 4 * seen * heads * hd}


# ----------------------------------------------------------------- inputs --
def _rope_table(n, hd):
    """(cos, sin) of position * theta^(-2 i / hd), [n][hd / 2][2] in fp32, from angles in 64 bits."""
    inv = THETA ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64, device="cuda") / hd)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.stack([a.cos(), a.sin()], dim=-1).float().contiguous()


def _inputs(case, seed):
    """The tensors of a case, made from its sizes and the seed."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    B = case["batch"]
    if case["op"] == "sample":
        V = case["vocab"]
        # a wide bulk, and a few tokens that the model favours
        logits = 2.0 * normal(B, V)
        at = (uniform(B, 64) * V).long().clamp(max=V - 1)
        logits.scatter_add_(1, at, 6.0 - 3.0 * torch.log(uniform(B, 64) + 1e-3))
        if case["masked"]:
            half = torch.arange(B, device="cuda")[:, None] % 2 == 0
            keep = uniform(B, V) < 0.05
            keep[:, 0] = True
            logits = torch.where(half & ~keep, -math.inf, logits)

        def choice(values):
            v = torch.tensor(values, device="cuda")
            return v[(uniform(B) * len(values)).long().clamp(max=len(values) - 1)]

        return {"logits": logits.to(dt), "u": uniform(B), "temperature": choice([0.7, 1.0, 1.0, 1.3]),
                "top_k": choice([20, 50, 1000, 0]).int() if case["top_k"] else None,
                "top_p": choice([0.9, 0.95, 0.5, 1.0]) if case["top_p"] else None,
                "min_p": choice([0.0, 0.02, 0.1]) if case["min_p"] else None}
    past, new = _lengths(case)
    kv, hd, page, nb = case["kv"], case["hd"], case["page"], _blocks(case)
    total = int(new.sum())
    s = {"pos": torch.from_numpy(past.astype(np.int32)).cuda(),
         "indptr": torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda(),
         "table": torch.rand(B * nb, generator=g, device="cuda").argsort().int().reshape(B, nb).contiguous(),
         "rope": _rope_table(case["past"] + case["new"], hd) if case["rope"] else None}
    channel = 0.5 + 1.5 * uniform(kv, hd)  # channels differ in size, as they do in a trained model
    if case["op"] == "append":
        s["k"] = (normal(total, kv, hd) * channel).to(dt)
        s["v"] = normal(total, kv, hd).to(dt)
        return s
    s["q"] = normal(total, kv * case["group"], hd).to(dt)
    # what the pages hold, new tokens included (they are appended before they are attended)
    s["k_pages"] = (normal(B * nb, page, kv, hd) * channel).to(dt)
    s["v_pages"] = normal(B * nb, page, kv, hd).to(dt)
    return s


# ----------------------------------------------------- the plain operators --
def _to_bf16(x):
    """x (64 bits) rounded to 8 significant bits, ties to even; scales stay far from the type's limits."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256.0) / 256.0, e)


def _down_to_bf16(x):
    m, e = torch.frexp(x)
    return torch.ldexp(torch.floor(m * 256.0) / 256.0, e)


def _quantise(x):
    """Codes, scales and offsets of the rows of x (64 bits: values lie next to the codes' borders)."""
    z = _down_to_bf16(x.amin(-1))
    s = _to_bf16((x.amax(-1) - z) / torch.full_like(z, 15.0))
    at = torch.where(s > 0, s, torch.ones_like(s))[..., None]
    c = torch.where(s[..., None] > 0, torch.round((x - z[..., None]) / at).clamp(0, 15), torch.zeros_like(x))
    return c.to(torch.uint8), s.float(), z.float()


def _rotate(x, cs):
    """Rows x [..., heads, hd] turned by the angles whose (cos, sin) are cs [..., hd / 2, 2]."""
    a, b = x.chunk(2, dim=-1)
    cos, sin = cs[..., 0].unsqueeze(-2), cs[..., 1].unsqueeze(-2)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _places(s, page, total):
    """Sequence, position, page and row in the page of each new token."""
    t = torch.arange(total, device="cuda")
    b = torch.searchsorted(s["indptr"][1:].contiguous(), t.int(), right=True)
    at = s["pos"][b].long() + t - s["indptr"][b]
    return b, at, s["table"][b, at // page].long(), at % page


def _plain_append(s):
    _, at, block, row = _places(s, s["page"], s["k"].shape[0])
    k, v = s["k"].double(), s["v"].double()
    if s["rope"] is not None:
        k = _rotate(k, s["rope"][at].double())
    out = []
    for x, held in ((k, s["held_k"]), (v, s["held_v"])):
        for part, value in zip(held, _quantise(x)):
            part[block, row] = value
        c, sc, z = (part[block, row] for part in held)
        out.append((c.float() * sc[..., None] + z[..., None]).to(s["k"].dtype))
    return {"k": out[0], "v": out[1]}


def _plain_attention(s):
    q, page, kv = s["q"], s["page"], s["kv"]
    total, heads, hd = q.shape
    b, at, _, _ = _places(s, page, total)
    x = q.float()
    if s["rope"] is not None:
        x = _rotate(x, s["rope"][at])
    B, nb = s["table"].shape
    k, v = ((c[s["table"].long()].float() * sc[s["table"].long()][..., None] + z[s["table"].long()][..., None])
            .reshape(B, nb * page, kv, hd) for c, sc, z in (s["held_k"], s["held_v"]))
    n = s["new"]
    i = torch.arange(total, device="cuda") - s["indptr"][b]
    padded = torch.zeros(B, n, heads, hd, device="cuda")
    padded[b, i] = x
    w = torch.matmul(padded.reshape(B, n, kv, heads // kv, hd).permute(0, 2, 3, 1, 4).reshape(B, kv, -1, hd),
                     k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(hd)).reshape(B, kv, heads // kv, n, nb * page)
    last = s["pos"].long()[:, None] + torch.arange(n, device="cuda")
    seen = torch.arange(nb * page, device="cuda")[None, None] <= last[..., None]
    w = w.masked_fill_(~seen[:, None, None], -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(w.reshape(B, kv, -1, nb * page), v.permute(0, 2, 1, 3)).reshape(B, kv, heads // kv, n, hd)
    o = o / w.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, heads, hd)[b, i].to(q.dtype)


def _plain_sample(s):
    """In 64 bits: long sums, and cumulated masses next to a border."""
    z = s["logits"].double()
    B, V = z.shape
    w = ((z - z.amax(-1, keepdim=True)) / s["temperature"].double()[:, None]).exp()
    _, order = torch.sort(s["logits"], dim=-1, descending=True, stable=True)
    ws = w.gather(1, order)
    rank = torch.arange(V, device="cuda")
    keep = z.gather(1, order) > -math.inf
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep = keep & ((rank < k) | (k <= 0))
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        cum = (ws * keep).cumsum(-1)
        before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], dim=-1)
        keep = keep & ((before < p * cum[:, -1:]) | (p >= 1))
    if s["min_p"] is not None:
        keep = keep & (ws >= s["min_p"].double()[:, None])
    kept = torch.zeros_like(keep).scatter(1, order, keep)
    cum = (w * kept).cumsum(-1)
    mass = cum[:, -1:]
    token = (cum <= s["u"].double()[:, None] * mass).sum(-1)
    token = torch.minimum(token, torch.where(kept, rank, -1).amax(-1))
    logprob = torch.log(w.gather(1, token[:, None]) / mass)[:, 0]
    return {"token": token.int(), "logprob": logprob.float(), "kept": kept.sum(-1).int()}


# -------------------------------------------------------------------- run --
def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "sample":
        return {**s, "op": "sample"}
    B, nb, page, kv, hd = case["batch"], _blocks(case), case["page"], case["kv"], case["hd"]
    s |= {"op": case["op"], "page": page, "kv": kv, "new": case["new"]}
    if own:
        from streaming_persistent_sm_b200 import wpk as W

        s["cache"] = W.KV4Cache(B * nb, kv, hd, page_tokens=page)
        if case["op"] == "attention":  # the pages, filled one by one as sequences of their own
            s["cache"].append(s.pop("k_pages").reshape(-1, kv, hd), s.pop("v_pages").reshape(-1, kv, hd),
                              torch.zeros(B * nb, dtype=torch.int32, device="cuda"),
                              torch.arange(B * nb, dtype=torch.int32, device="cuda")[:, None].contiguous())
        return s

    def empty():
        return (torch.zeros(B * nb, page, kv, hd, dtype=torch.uint8, device="cuda"),
                torch.zeros(B * nb, page, kv, device="cuda"), torch.zeros(B * nb, page, kv, device="cuda"))

    if case["op"] == "append":
        s["held_k"], s["held_v"] = empty(), empty()
    else:
        s["held_k"] = _quantise(s.pop("k_pages").double())
        s["held_v"] = _quantise(s.pop("v_pages").double())
    return s


def run(s):
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "sample": _plain_sample}[s["op"]](s)
    from streaming_persistent_sm_b200 import wpk as W

    if s["op"] == "append":
        s["cache"].append(s["k"], s["v"], s["pos"], s["table"], indptr=s["indptr"], rope=s["rope"])
        k, v = s["cache"].read(s["pos"], s["table"], s["k"].shape[0], indptr=s["indptr"], dtype=s["k"].dtype)
        return {"k": k, "v": v}
    if s["op"] == "attention":
        return s["cache"].attention(s["q"], s["pos"], s["table"], indptr=s["indptr"], max_new=s["new"], rope=s["rope"])
    token, logprob, kept = W.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                    top_p=s["top_p"], min_p=s["min_p"], want_logprob=True, want_kept=True)
    return {"token": token, "logprob": logprob, "kept": kept}


# ------------------------------------------------------------------ exact --
def _held(x):
    """The values that the cache holds for rows x, in 64 bits.  A bf16 number is a multiple of 2^(e - 7)
    for 2^e <= |x| < 2^(e + 1)."""
    def unit(y):
        return torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1e-300))) - 7)

    lo, hi = x.min(dim=-1, keepdim=True).values, x.max(dim=-1, keepdim=True).values
    z = torch.floor(lo / unit(lo)) * unit(lo)
    step = (hi - z) / torch.tensor(15.0, dtype=torch.float64, device=x.device).expand_as(z)
    s = torch.round(step / unit(step)) * unit(step)
    c = torch.round((x - z) / s.clamp(min=1e-300)).clamp(min=0, max=15)
    return torch.where(s == 0, z, c * s + z)


def _turned(x, at, hd, angles):
    """x [n, heads, hd] rotated to positions at: pair (i, i + hd / 2) as one complex number.  The angles'
    cosines and sines are an input of the operator, in fp32."""
    w = torch.view_as_complex(angles[at].double().contiguous())[:, None]
    y = torch.complex(x[..., : hd // 2], x[..., hd // 2:]) * w
    return torch.cat([y.real, y.imag], dim=-1)


def _exact_sample(case, s):
    z = s["logits"].double().cpu().numpy()
    T, u = s["temperature"].double().cpu().numpy(), s["u"].double().cpu().numpy()
    get = lambda n, d: s[n].double().cpu().numpy() if s[n] is not None else np.full(len(u), d)  # noqa: E731
    ks, ps, ms = get("top_k", 0), get("top_p", 1.0), get("min_p", 0.0)
    logprob = np.empty(len(u))
    for r in range(len(u)):
        ids = np.flatnonzero(z[r] > -np.inf)
        order = ids[np.argsort(-z[r][ids], kind="stable")]
        w = np.exp((z[r][order] - z[r].max()) / T[r])
        if ks[r] > 0:
            order, w = order[: int(ks[r])], w[: int(ks[r])]
        if ps[r] < 1:
            n = int(np.searchsorted(np.cumsum(w), ps[r] * w.sum(), side="left")) + 1
            order, w = order[:n], w[:n]
        order, w = order[w >= ms[r]], w[w >= ms[r]]
        by_id = np.argsort(order)
        cum = np.cumsum(w[by_id])
        j = min(int(np.searchsorted(cum, u[r] * cum[-1], side="right")), len(cum) - 1)
        logprob[r] = np.log(w[by_id[j]]) - np.log(cum[-1])
    return {"token": None, "logprob": torch.from_numpy(logprob), "kept": None}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "sample":
        return _exact_sample(case, s)
    hd, kv, page = case["hd"], case["kv"], case["page"]
    past, new = _lengths(case)
    at = torch.cat([torch.arange(p, p + n, device="cuda") for p, n in zip(past.tolist(), new.tolist())])
    if case["op"] == "append":
        k = s["k"].double()
        return {"k": _held(k if s["rope"] is None else _turned(k, at, hd, s["rope"])), "v": _held(s["v"].double())}
    q = s["q"].double()
    if s["rope"] is not None:
        q = _turned(q, at, hd, s["rope"])
    out, first = torch.empty_like(q), 0
    for b in range(case["batch"]):
        p, n = int(past[b]), int(new[b])
        pages = s["table"][b, : -(-(p + n) // page)].long()
        k, v = (_held(s[x][pages].double()).reshape(-1, kv, hd)[: p + n] for x in ("k_pages", "v_pages"))
        x = q[first:first + n].reshape(n, kv, case["group"], hd)
        a = torch.einsum("nkgd,skd->kgns", x, k) / math.sqrt(hd)
        later = torch.arange(p + n, device="cuda")[None] > torch.arange(p, p + n, device="cuda")[:, None]
        a = torch.softmax(a.masked_fill(later, -math.inf), dim=-1)
        out[first:first + n] = torch.einsum("kgns,skd->nkgd", a, v).reshape(n, -1, hd)
        first += n
    return out
