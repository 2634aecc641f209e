"""Serving from a paged cache: the two operators, what they are measured on, and their plain forms.

One serving step takes new tokens of b sequences, packed one sequence after another (q_starts[s] is the first
row of sequence s), and caches whose keys and values lie in pages [n_pages, h_kv, page, d] that a table
[b, pages_per_seq] assigns to the sequences.  kv_lengths[s] counts the positions of sequence s, its new tokens
included, so new token i of n sits at position kv_lengths[s] - n + i.
  append     rotates the new queries and keys by their positions and stores keys and values into the pages
  attention  softmax(scale q k^T) v of each new token over its sequence's positions up to its own; query
             head x reads key-value head x // (h / h_kv)

Head shapes are the base model's (64 wide, 8 heads), the big model's (64 wide, 16 heads) and the long causal
workload's (128 wide, 16 heads), with as many or fewer key-value heads; caches go up to that workload's 8192
positions and far beyond it for one sequence.
"""
import math

import torch

own = False


def _case(name, op, b, prompts, new_lo, new_hi, len_lo, len_hi, h, h_kv, d, page, d_rot=0, interleaved=False,
          packed=False):
    c = {"op": op, "b": b, "prompts": prompts, "new_lo": new_lo, "new_hi": new_hi, "len_lo": len_lo,
         "len_hi": len_hi, "h": h, "h_kv": h_kv, "d": d, "page": page, "d_rot": d_rot,
         "interleaved": interleaved, "packed": packed}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token for each of 8 chats with a base model: the launch is all there is
        _case("append_step_b8", "append", 8, 0, 1, 1, 20, 500, 8, 8, 64, 16, 64),
        # one token for each of 256 sequences, grouped heads
        _case("append_step_b256", "append", 256, 0, 1, 1, 300, 500, 16, 4, 128, 64, 128),
        # odd prompts of a few hundred tokens, half of each head rotated in neighbouring pairs, rows cut out of
        # the packed result of one projection
        _case("append_ragged", "append", 7, 7, 33, 601, 0, 900, 16, 16, 64, 32, 32, True, True),
        # two prompts of 8192 tokens
        _case("append_prompt", "append", 2, 2, 8192, 8192, 0, 0, 16, 4, 128, 64, 128, False, True),
        # one token of one short chat: latency
        _case("step_b1_short", "attention", 1, 0, 1, 1, 300, 300, 8, 8, 64, 16),
        # one token for each of 32 sequences over 4096 to 8192 cached positions
        _case("step_b32", "attention", 32, 0, 1, 1, 4096, 8192, 16, 4, 128, 64),
        # one sequence of 131072 positions
        _case("step_long", "attention", 1, 0, 1, 1, 131072, 131072, 16, 2, 128, 64),
        # four drafted tokens to verify for each of 16 sequences, a key-value head for each query head
        _case("verify_b16", "attention", 16, 16, 4, 4, 1000, 4001, 16, 16, 64, 32),
        # chunks of 512 prompt tokens behind 7680 cached positions
        _case("chunk_b4", "attention", 4, 4, 512, 512, 8192, 8192, 16, 4, 128, 64),
        # whole prompts of 8192 tokens
        _case("prompt_b2", "attention", 2, 2, 8192, 8192, 0, 0, 16, 4, 128, 64),
        # two odd prompts among single tokens, three query heads to a key-value head, small pages
        _case("mixed_b24", "attention", 24, 2, 301, 1501, 60, 5001, 24, 8, 64, 16),
        # wide heads, a chunk of 200 behind 2800 positions, one key-value head
        _case("chunk_wide", "attention", 3, 3, 200, 200, 2999, 2999, 8, 1, 256, 128),
    ]


def _spread(i, lo, hi, step):
    return lo + int((hi - lo + 1) * ((i * step + 0.37) % 1.0))


def _sizes(c):
    """New tokens and lengths of each sequence: a fixed spread over the case's ranges."""
    new, lens = [], []
    for i in range(c["b"]):
        n = _spread(i, c["new_lo"], c["new_hi"], 0.618034) if i < c["prompts"] else 1
        new.append(n)
        lens.append(max(n, _spread(i, c["len_lo"], c["len_hi"], 0.754878)))
    return new, lens


def _pairs(c):
    """Visible (token, key) pairs of one head."""
    return sum(n * (s - n) + n * (n + 1) // 2 for n, s in zip(*_sizes(c)))


def _padded(c):
    new, lens = _sizes(c)
    return c["b"] * c["h"] * max(new) * max(lens)


def work(case):
    c = case
    new, lens = _sizes(c)
    t, h, h_kv, d = sum(new), c["h"], c["h_kv"], c["d"]
    if c["op"] == "append":
        rotated = t * (h + h_kv) * c["d_rot"]
        return {"bytes": 2 * t * (h + 2 * h_kv) * d * 2 + 4 * (t + 2 * c["b"]), "flops": 3 * rotated}
    return {"bytes": 2 * t * h * d * 2 + 2 * sum(lens) * h_kv * d * 2 + 4 * sum(-(-s // c["page"]) for s in lens),
            "flops": 4 * d * h * _pairs(c)}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_padded(c) for c in listed() if c["op"] == "attention")
    top = {op: [max(work(c)[k] for c in listed() if c["op"] == op) for k in ("bytes", "flops")]
           for op in ("append", "attention")}
    while True:
        op = rng.choice(["append", "attention", "attention"])
        h_kv, group, d = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([32, 64, 64, 128, 128, 256])
        b = _log(rng, 1, 128)
        kind = rng.choice(["step", "few", "chunk", "mixed"])
        new_hi = {"step": 1, "few": rng.randint(2, 8), "chunk": _log(rng, 9, 8192), "mixed": _log(rng, 9, 2048)}[kind]
        new_lo = rng.randint(1, new_hi)
        prompts = {"step": 0, "few": b, "chunk": b, "mixed": max(1, b // 8)}[kind]
        len_hi = _log(rng, max(1, new_hi // 2), 131072)
        c = _case(None, op, b, prompts, new_lo, new_hi, rng.randint(1, len_hi), len_hi, h_kv * group, h_kv, d,
                  rng.choice([16, 32, 64, 128, 256]))
        if op == "append":
            c["d_rot"] = rng.choice([0, 16, d // 2, d, d])
            c["interleaved"], c["packed"] = rng.random() < 0.5, rng.random() < 0.5
            c["len_lo"], c["len_hi"] = min(c["len_lo"], 2000), min(c["len_hi"], 2000)
        w = work(c)
        cached = sum(_sizes(c)[1]) * h_kv * d
        if (c["h"] <= 64 and cached <= 1 << 28 and w["bytes"] <= top[op][0] and w["flops"] <= top[op][1]
                and (op == "append" or _padded(c) <= most)):
            return c


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    new, lens = _sizes(c)
    b, t, h, h_kv, d, page = c["b"], sum(new), c["h"], c["h_kv"], c["d"], c["page"]
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    # pages are handed out in no order; entries past a sequence's last page are never read
    need = [-(-s // page) for s in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((b, max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    starts = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    s = {"case": c, "max_new": max(new), "table": table.to(dev), "starts": starts.to(dev),
         "lengths": torch.tensor(lens, dtype=torch.int32, device=dev),
         "k_pages": normal(n_pages, h_kv, page, d), "v_pages": normal(n_pages, h_kv, page, d)}
    if c["op"] == "append":
        if c["packed"]:   # [t, (h + 2 h_kv) d], the rows of one projection
            rows = normal(t, h + 2 * h_kv, d)
            s["q"], s["k"], s["v"] = rows[:, :h], rows[:, h:h + h_kv], rows[:, h + h_kv:]
        else:
            s["q"], s["k"], s["v"] = normal(t, h, d), normal(t, h_kv, d), normal(t, h_kv, d)
        if c["d_rot"]:
            i = torch.arange(0, c["d_rot"], 2, dtype=torch.float64)
            s["freqs"] = (10000.0 ** (-i / c["d_rot"])).float().to(dev)
        else:
            s["freqs"] = None
        s["q_out"] = torch.empty(t, h, d, dtype=torch.bfloat16, device=dev)
    else:
        s["q"] = normal(t, h, d)
        s["out"] = torch.empty(t, h, d, dtype=torch.bfloat16, device=dev)
    return s


def _tokens(s):
    """Sequence and position of every packed token."""
    starts = s["starts"].long()
    t = torch.arange(s["q"].shape[0], device=starts.device)
    seq = torch.searchsorted(starts, t, right=True) - 1
    return seq, s["lengths"].long()[seq] - starts[seq + 1] + t


def _rotate(x, cos, sin, interleaved):
    n = 2 * cos.shape[-1]
    if not n:
        return x
    x, y = x.float(), x
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if interleaved else (x[..., :n // 2], x[..., n // 2:n])
    p, q = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((p, q), -1).flatten(-2) if interleaved else torch.cat((p, q), -1)
    return torch.cat((r.to(y.dtype), y[..., n:]), -1)


def _plain_append(s):
    c = s["case"]
    seq, pos = _tokens(s)
    n = c["d_rot"] // 2
    # angles of far positions need 64 bits
    angle = pos.double()[:, None, None] * (s["freqs"].double() if n else pos.new_zeros(0).double())
    cos, sin = angle.cos().float(), angle.sin().float()
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["interleaved"]))
    at = s["table"][seq, pos // c["page"]].long()
    s["k_pages"][at, :, pos % c["page"]] = _rotate(s["k"], cos, sin, c["interleaved"])
    s["v_pages"][at, :, pos % c["page"]] = s["v"]
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attention(s):
    c = s["case"]
    b, h_kv, d, n = c["b"], c["h_kv"], c["d"], s["max_new"]
    g = c["h"] // h_kv
    starts, lens = s["starts"].long(), s["lengths"].long()
    new = starts[1:] - starts[:-1]
    at = s["table"].long().clamp(min=0)

    def cached(pages):   # [b, h_kv, positions, d]
        return pages[at].transpose(1, 2).flatten(2, 3).float()

    i = torch.arange(n, device=at.device)
    q = s["q"][(starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].float()         # [b, n, h, d]
    q = q.view(b, n, h_kv, g, d).permute(0, 2, 3, 1, 4).reshape(b, h_kv, g * n, d)
    x = torch.matmul(q, cached(s["k_pages"]).transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    j = torch.arange(x.shape[-1], device=at.device)
    seen = j <= ((lens - new)[:, None] + i)[..., None]                                  # [b, n, positions]
    x = x.view(b, h_kv, g, n, -1).masked_fill_(~seen[:, None, None], -math.inf)
    p = torch.exp(x.sub_(x.amax(-1, keepdim=True).clamp(min=-3e38)))
    p = torch.where(seen[:, None, None], p, 0.0)
    v = torch.where((j < lens[:, None])[:, None, :, None], cached(s["v_pages"]), 0.0)
    o = torch.matmul(p.view(b, h_kv, g * n, -1), v) / p.sum(-1).clamp(min=1e-30).view(b, h_kv, g * n, 1)
    o = o.view(b, h_kv * g, n, d)
    seq, pos = _tokens(s)
    s["out"].copy_(o[seq, :, pos - (lens - new)[seq]])
    return {"out": s["out"]}


def run(state):
    s = state
    if not own:
        return _plain_append(s) if s["case"]["op"] == "append" else _plain_attention(s)
    import transformer_scaled_dot_02_gb300 as sd
    if s["case"]["op"] == "append":
        sd.paged_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["starts"], s["lengths"],
                        rope_freqs=s["freqs"], interleaved=s["case"]["interleaved"], q_out=s["q_out"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if "workspace" not in s:   # a serving loop keeps one
        s["workspace"] = sd.paged_workspace(s["q"], s["k_pages"], s["table"])
    sd.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["starts"], s["lengths"], out=s["out"],
                       workspace=s["workspace"])
    return {"out": s["out"]}


def exact(case, seed):
    """The definitions, sequence by sequence and in 64 bits."""
    s = prepare(case, seed)
    c = case
    new, lens = _sizes(c)
    h, h_kv, d, page = c["h"], c["h_kv"], c["d"], c["page"]
    table = s["table"].cpu().tolist()
    if c["op"] == "append":
        q, kp, vp = s["q"].double(), s["k_pages"].double(), s["v_pages"].double()
        k, v = s["k"].double(), s["v"].double()
        t = 0
        for n, length, pages in zip(new, lens, table):
            pos = torch.arange(length - n, length, device=q.device)
            rows = slice(t, t + n)
            if c["d_rot"]:
                turn = torch.polar(torch.ones((), dtype=torch.float64, device=q.device),
                                   pos.double()[:, None] * s["freqs"].double())[:, None]
                for x in (q, k):
                    part = x[rows, :, :c["d_rot"]]
                    if c["interleaved"]:
                        z = torch.complex(part[..., 0::2], part[..., 1::2]) * turn
                        part[..., 0::2], part[..., 1::2] = z.real, z.imag
                    else:
                        m = c["d_rot"] // 2
                        z = torch.complex(part[..., :m], part[..., m:]) * turn
                        part[..., :m], part[..., m:] = z.real, z.imag
            at = torch.tensor(pages, device=q.device)[pos // page]
            kp[at, :, pos % page], vp[at, :, pos % page] = k[rows], v[rows]
            t += n
        return {"q": q, "k_pages": kp, "v_pages": vp}
    out = torch.empty(sum(new), h, d, dtype=torch.float64, device=s["q"].device)
    t = 0
    for n, length, pages in zip(new, lens, table):
        at = torch.tensor(pages[:-(-length // page)], device=out.device)
        pos = torch.arange(length - n, length, device=out.device)
        hidden = torch.arange(length, device=out.device)[None] > pos[:, None]
        for x in range(h):
            y = x // (h // h_kv)
            k = s["k_pages"][at, y].reshape(-1, d)[:length].double()
            v = s["v_pages"][at, y].reshape(-1, d)[:length].double()
            w = s["q"][t:t + n, x].double() @ k.T / math.sqrt(d)
            out[t:t + n, x] = torch.softmax(w.masked_fill(hidden, -math.inf), -1) @ v
        t += n
    return {"out": out}
