"""The serving operators as measured cases: token sampling, the paged key/value cache with its append and its
one-token attention, and the attention of packed prompts.

Each case has a plain form (elementary torch operations in 32 bits, in 64 where angles, sums or borders need them)
and the call a program makes of the library.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
DT = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # the audio heads of two sessions' 8 agent codebooks, at the model's default sampling: latency counts
        dict(name="sample_audio", op="sample", rows=16, cols=2048, dtype=F32, mode="topk", k=250, t=0.8, spread=2.0),
        # the text head of a batch of sessions at its default sampling
        dict(name="sample_text", op="sample", rows=32, cols=32000, dtype=F32, mode="topk", k=25, t=0.7, spread=3.0),
        # nucleus sampling for a large batch, no top-k to narrow the row first
        dict(name="sample_nucleus", op="sample", rows=256, cols=32000, dtype=F32, mode="nucleus", k=0, t=1.0, spread=3.0),
        # a large odd vocabulary in 16 bits (many equal logits), every request with settings of its own
        dict(name="sample_mixed", op="sample", rows=128, cols=131071, dtype=BF16, mode="mixed", k=0, t=1.0, spread=3.0),
        # one new frame of each of four sessions, in the parity type: latency counts
        dict(name="append_step", op="append", seqs=4, tokens=4, hq=16, hkv=16, hd=64, page=16, dtype=F32, rope="interleaved", far=3000),
        # packed prompts of uneven length entering the cache, grouped heads, half-split rotation
        dict(name="append_prompt", op="append", seqs=7, tokens=8192, hq=32, hkv=8, hd=128, page=16, dtype=BF16, rope="half", far=65536),
        # one session's frame over a full ring's worth of keys: the B = 1 latency case
        dict(name="decode_one", op="decode", seqs=1, len=3000, hq=32, hkv=32, hd=128, page=64, dtype=BF16, window=0, ragged=False),
        # a serving batch of uneven lengths, grouped heads, small pages
        dict(name="decode_batch", op="decode", seqs=32, len=8192, hq=32, hkv=8, hd=128, page=16, dtype=BF16, window=0, ragged=True),
        # few long contexts: the work has to be split over the length
        dict(name="decode_long", op="decode", seqs=4, len=131072, hq=64, hkv=8, hd=128, page=128, dtype=BF16, window=0, ragged=True),
        # a persona prompt of one session
        dict(name="prompt_persona", op="prompt", seqs=1, tokens=137, hq=32, hkv=32, hd=128, dtype=BF16, window=0),
        # packed prompts of uneven length, grouped heads
        dict(name="prompt_packed", op="prompt", seqs=12, tokens=8192, hq=32, hkv=8, hd=128, dtype=BF16, window=0),
        # one prompt as long as the context
        dict(name="prompt_long", op="prompt", seqs=1, tokens=8192, hq=32, hkv=8, hd=128, dtype=BF16, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "append", "decode", "prompt"])
    if op == "sample":
        rows, cols = _log(rng, 1, 256), _log(rng, 100, 131072)
        mode = rng.choice(["topk", "nucleus", "mixed"])
        rows = min(rows, 16_000_000 // cols)
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice([F32, F32, BF16]), mode=mode,
                    k=_log(rng, 1, 2000) if mode == "topk" else 0, t=round(rng.uniform(0.3, 1.5), 2), spread=round(rng.uniform(1.0, 4.0), 2))
    hkv, g = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 3, 4, 6, 8])
    while hkv * g > 64:
        g = rng.choice([1, 2, 3, 4, 6, 8])
        hkv = rng.choice([1, 2, 4, 8, 16, 32])
    hd, dtype = rng.choice([64, 128]), rng.choice([BF16, BF16, F32])
    if op == "append":
        tokens = _log(rng, 1, 8192)
        if tokens * hkv * (g + 2) * hd * (2 if dtype == BF16 else 4) > 100_000_000:
            tokens = max(1, tokens // 8)
        return dict(op=op, seqs=min(tokens, _log(rng, 1, 64)), tokens=tokens, hq=hkv * g, hkv=hkv, hd=hd,
                    page=rng.choice([1, 16, 32, 48, 64, 128]), dtype=dtype, rope=rng.choice(["interleaved", "half"]), far=_log(rng, 100, 131072))
    if op == "decode":
        seqs, length = _log(rng, 1, 64), _log(rng, 16, 65536)
        while 2 * seqs * length * hkv * hd * (2 if dtype == BF16 else 4) > 1_200_000_000:
            length = max(16, length // 2)
            seqs = max(1, seqs // 2)
        return dict(op=op, seqs=seqs, len=length, hq=hkv * g, hkv=hkv, hd=hd, page=rng.choice([1, 16, 32, 48, 64, 128]), dtype=dtype,
                    window=rng.choice([0, 0, 1000, 3000 - 1]), ragged=rng.random() < 0.7)
    tokens = _log(rng, 1, 8192)
    if dtype == F32:
        tokens = min(tokens, 2048 + tokens // 8)
    while tokens * tokens * hkv * g > 8192 * 8192 * 16:
        tokens //= 2
    return dict(op=op, seqs=min(tokens, _log(rng, 1, 24)), tokens=tokens, hq=hkv * g, hkv=hkv, hd=hd, dtype=dtype,
                window=rng.choice([0, 0, 500, 2999]))


def _lengths(case):
    """Uneven lengths of at least one token, in no order, that add up to the case's tokens."""
    r = np.random.RandomState(case["tokens"])
    n, total = case["seqs"], case["tokens"]
    w = np.linspace(1.0, 4.0, n) if n > 1 else np.ones(1)
    lens = np.maximum(1, np.floor(total * w / w.sum())).astype(np.int64)
    lens[-1] += total - lens.sum()
    while lens[-1] < 1:
        lens[np.argmax(lens)] -= 1
        lens[-1] += 1
    r.shuffle(lens)
    return [int(x) for x in lens]


def _kv_lengths(case):
    n = case["seqs"]
    if not case["ragged"] or n == 1:
        return [case["len"]] * n
    return [max(1, int(case["len"] * (i + 1) / n) - (i * 7) % 13) for i in range(n)]


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _pages(case, lens, gen, dev):
    """A table of distinct pages in a shuffled pool, as many as the lengths need; unused entries are -1."""
    page = case["page"]
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need), generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return sum(need), table


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(0.0, scale, generator=gen)

    s = dict(case)
    if case["op"] == "sample":
        n, c = case["rows"], case["cols"]
        s["logits"] = normal(n, c, scale=case["spread"]).to(DT[case["dtype"]])
        s["u"] = torch.rand(n, generator=gen, device=dev)
        mode = case["mode"]
        t = torch.full((n,), case["t"], device=dev)
        k = torch.full((n,), case["k"], dtype=torch.int32, device=dev)
        p, m = torch.ones(n, device=dev), torch.zeros(n, device=dev)
        if mode == "nucleus":
            p.fill_(0.9)
            m.fill_(0.001)
        elif mode == "mixed":  # rows in turn: greedy, top-k, top-p, min-p, all three, nothing but the temperature
            i = torch.arange(n, device=dev)
            t = torch.where(i % 6 == 0, torch.zeros_like(t), t * (0.7 + 0.1 * (i % 5).float()))
            k = torch.where((i % 6 == 1) | (i % 6 == 4), 20 + 30 * (i % 11), torch.zeros_like(i)).to(torch.int32)
            p = torch.where((i % 6 == 2) | (i % 6 == 4), 0.8 + 0.03 * (i % 7).float(), p)
            m = torch.where((i % 6 == 3) | (i % 6 == 4), 0.01 + 0.01 * (i % 5).float(), m)
        s.update(t_row=t.float(), k_row=k, p_row=p.float(), m_row=m.float(), out=torch.empty(n, dtype=torch.int32, device=dev))
        return s
    dt, hq, hkv, hd = DT[case["dtype"]], case["hq"], case["hkv"], case["hd"]
    if case["op"] == "append":
        lens = _lengths(case)
        n = sum(lens)
        past = np.random.RandomState(case["far"]).randint(0, case["far"], len(lens)).tolist()
        total = [a + b for a, b in zip(past, lens)]
        qkv = normal(n, hq + 2 * hkv, hd).to(dt)  # one projection's output: the three parts are strided views of it
        s.update(lens=lens, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], cu=_i32(np.cumsum([0] + lens).tolist(), dev), kv_len=_i32(total, dev))
        # the pool holds the pages that the new tokens reach, and the table names only those
        page = case["page"]
        first = [a // page for a in past]
        need = [-(-b // page) - a for a, b in zip(first, total)]
        order = torch.randperm(sum(need), generator=gen, device=dev).to(torch.int32)
        table = torch.full((len(lens), max(-(-b // page) for b in total)), -1, dtype=torch.int32, device=dev)
        at = 0
        for i, c in enumerate(need):
            table[i, first[i]:first[i] + c] = order[at:at + c]
            at += c
        s["table"] = table
        s["kc"], s["vc"] = normal(sum(need), hkv, page, hd).to(dt), normal(sum(need), hkv, page, hd).to(dt)
        s["q_out"], s["k_out"] = torch.empty(n, hq, hd, dtype=dt, device=dev), torch.empty(n, hkv, hd, dtype=dt, device=dev)
    elif case["op"] == "decode":
        lens = _kv_lengths(case)
        pages, s["table"] = _pages(case, lens, gen, dev)
        s["kc"], s["vc"] = normal(pages, hkv, case["page"], hd, dtype=dt), normal(pages, hkv, case["page"], hd, dtype=dt)
        s.update(lens=lens, kv_len=_i32(lens, dev), q=normal(len(lens), hq, hd, dtype=dt), out=torch.empty(len(lens), hq, hd, dtype=dt, device=dev))
    else:
        lens = _lengths(case)
        n = sum(lens)
        s.update(lens=lens, cu=_i32(np.cumsum([0] + lens).tolist(), dev), q=normal(n, hq, hd, dtype=dt), k=normal(n, hkv, hd, dtype=dt),
                 v=normal(n, hkv, hd, dtype=dt), out=torch.empty(n, hq, hd, dtype=dt, device=dev))
    if own and "kc" in s:
        from full_duplex_speech_frame_gb300 import mfs
        s["cache"] = mfs.PagedKV(s["kc"], s["vc"], s["table"])
        if case["op"] == "decode":
            s["workspace"] = mfs.mfs_paged_attention_workspace(s["cache"], hq)
    return s


def run(state):
    return {"sample": _sample, "append": _append, "decode": _decode, "prompt": _prompt}[state["op"]](state)


def _sample(s):
    if own:
        from full_duplex_speech_frame_gb300 import mfs
        mfs.mfs_sample_rows(s["logits"], s["u"], s["out"], temperature=s["t_row"], top_k=s["k_row"], top_p=s["p_row"], min_p=s["m_row"])
        return s["out"]
    # 64 bits: a token is drawn at a border of the running sum
    x, index = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    c = x.shape[1]
    t = s["t_row"].double()[:, None]
    d = x.double() - x[:, :1].double()
    w = torch.exp(d / torch.where(t > 0, t, torch.ones_like(t)))
    rank = torch.arange(c, device=x.device)[None]
    k = torch.where(s["k_row"] > 0, s["k_row"].long().clamp(max=c), torch.full_like(s["k_row"], c).long())[:, None]
    k = torch.where(t > 0, k, torch.ones_like(k))
    w = torch.where((rank < k) & (w >= s["m_row"].double()[:, None]), w, torch.zeros_like(w))
    run_sum = torch.cumsum(w, 1)
    p = s["p_row"].double()[:, None]
    before = run_sum - w  # the first candidate stays; another one stays while those before it hold less than p
    keep = (rank == 0) | (p >= 1) | (before < p * run_sum[:, -1:])
    w = torch.where(keep, w, torch.zeros_like(w))
    in_order = torch.zeros_like(w).scatter_(1, index, w)
    run_sum = torch.cumsum(in_order, 1)
    return (run_sum > s["u"].double()[:, None] * run_sum[:, -1:]).to(torch.int8).argmax(1).to(torch.int32)


def _rotate(x, angle, rope):
    """x [N, H, hd] by angle [N, hd / 2] (64 bits), in 32 bits."""
    c, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    x = x.float()
    if rope == "half":
        a, b = x.chunk(2, dim=-1)
        return torch.cat([a * c - b * sn, a * sn + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)


def _append(s):
    if own:
        from full_duplex_speech_frame_gb300 import mfs
        mfs.mfs_kv_append(s["cache"], s["k"], s["v"], s["cu"], s["kv_len"], q=s["q"], q_out=s["q_out"], k_out=s["k_out"], rope=s["rope"], theta=10000.0)
        return s["q_out"], s["k_out"], s["kc"], s["vc"]
    n, hd = s["k"].shape[0], s["hd"]
    tok = torch.arange(n, device=s["k"].device)
    seq = torch.bucketize(tok, s["cu"][1:].long(), right=True)
    pos = s["kv_len"].long()[seq] - s["cu"].long()[seq + 1] + tok
    freq = 10000.0 ** (-2.0 * torch.arange(hd // 2, device=pos.device, dtype=torch.float64) / hd)
    angle = pos.double()[:, None] * freq
    dt = s["k"].dtype
    s["q_out"].copy_(_rotate(s["q"], angle, s["rope"]).to(dt))
    s["k_out"].copy_(_rotate(s["k"], angle, s["rope"]).to(dt))
    page, row = s["table"].long()[seq, pos // s["page"]], pos % s["page"]
    s["kc"][page, :, row] = s["k_out"]
    s["vc"][page, :, row] = s["v"]
    return s["q_out"], s["k_out"], s["kc"], s["vc"]


def _decode(s):
    if own:
        from full_duplex_speech_frame_gb300 import mfs
        mfs.mfs_paged_attention(s["cache"], s["q"], s["kv_len"], s["out"], window=s["window"], workspace=s["workspace"])
        return s["out"]
    n, hkv, hd = len(s["lens"]), s["hkv"], s["hd"]
    longest = max(s["lens"])
    first = max(0, min(s["lens"]) - s["window"]) if s["window"] else 0
    pos = torch.arange(first, longest, device=s["q"].device)
    length = s["kv_len"].long()[:, None]
    seen = pos[None] < length
    if s["window"]:
        seen = seen & (pos[None] >= length - s["window"])
    page = s["table"].long()[:, pos // s["page"]].clamp(min=0)
    row = (pos % s["page"])[None].expand_as(page)
    k = s["kc"][page, :, row].float().permute(0, 2, 1, 3)  # [n, hkv, L, hd]
    q = s["q"].float().view(n, hkv, -1, hd)
    a = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(hd))
    del k
    seen = seen[:, None, None]
    a = torch.where(seen, a, torch.full_like(a, -math.inf))
    a = torch.where(seen, torch.exp(a - a.amax(-1, keepdim=True)), torch.zeros_like(a))
    a = a / a.sum(-1, keepdim=True)
    v = s["vc"][page, :, row].float().permute(0, 2, 1, 3)
    return torch.matmul(a, v).reshape(n, -1, hd).to(s["q"].dtype)


def _prompt(s):
    if own:
        from full_duplex_speech_frame_gb300 import mfs
        mfs.mfs_prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["out"], window=s["window"])
        return s["out"]
    hq, hkv, hd = s["hq"], s["hkv"], s["hd"]
    longest = max(s["lens"])
    at = torch.arange(longest, device=s["q"].device)
    length = (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    inside = at[None] < length  # [n, L]: the sequences side by side, short ones padded with their first token
    tok = s["cu"][:-1].long()[:, None] + torch.where(inside, at[None], torch.zeros_like(at)[None])
    q = s["q"][tok].float().view(len(s["lens"]), longest, hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4)
    k = s["k"][tok].float().permute(0, 2, 3, 1)[:, :, None]
    a = torch.matmul(q, k) * (1.0 / math.sqrt(hd))
    seen = at[None] <= at[:, None]
    if s["window"]:
        seen = seen & (at[None] > at[:, None] - s["window"])
    a = torch.where(seen, a, a.new_full((), -math.inf))
    a = torch.exp(a - a.amax(-1, keepdim=True))
    a = a / a.sum(-1, keepdim=True)
    v = s["v"][tok].float().permute(0, 2, 1, 3)[:, :, None]
    o = torch.matmul(a, v).permute(0, 3, 1, 2, 4).reshape(len(s["lens"]), longest, hq, hd)
    return o[inside].to(s["q"].dtype)


def work(case):
    if case["op"] == "sample":
        return {"bytes": case["rows"] * (case["cols"] * (4 if case["dtype"] == F32 else 2) + 24), "flops": 0}
    e = 2 if case["dtype"] == BF16 else 4
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    if case["op"] == "append":  # q in and out; k in, out and into the cache; v in and into the cache
        return {"bytes": case["tokens"] * hd * e * (2 * hq + 5 * hkv), "flops": 3 * case["tokens"] * hd * (hq + hkv)}
    if case["op"] == "decode":
        keys = sum(min(n, case["window"]) if case["window"] else n for n in _kv_lengths(case))
        return {"bytes": e * hd * (2 * keys * hkv + 2 * case["seqs"] * hq) + 4 * case["seqs"], "flops": 4 * keys * hq * hd}
    w, pairs = case["window"], 0
    for n in _lengths(case):
        m = min(n, w) if w else n
        pairs += m * (m + 1) // 2 + (n - m) * m
    return {"bytes": case["tokens"] * hd * e * (2 * hq + 2 * hkv), "flops": 4 * pairs * hq * hd}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    hd, page = case["hd"], case.get("page")
    if case["op"] == "append":
        q, k, v = (s[x].cpu().double().numpy() for x in "qkv")
        table, kc, vc = s["table"].cpu().numpy(), s["kc"].cpu().double().numpy(), s["vc"].cpu().double().numpy()
        freq = np.power(10000.0, -2.0 * np.arange(hd // 2) / hd)
        x, y = (np.arange(0, hd, 2), np.arange(1, hd, 2)) if case["rope"] == "interleaved" else (np.arange(hd // 2), np.arange(hd // 2, hd))
        q_out, k_out = np.empty_like(q), np.empty_like(k)
        t = 0
        for i, n in enumerate(s["lens"]):
            for p in range(int(s["kv_len"][i]) - n, int(s["kv_len"][i])):
                turn = np.exp(1j * p * freq)
                for src, dst in ((q, q_out), (k, k_out)):
                    z = (src[t][:, x] + 1j * src[t][:, y]) * turn
                    dst[t][:, x], dst[t][:, y] = z.real, z.imag
                kc[table[i, p // page], :, p % page] = k_out[t]
                vc[table[i, p // page], :, p % page] = v[t]
                t += 1
        return q_out, k_out, kc, vc
    hq, hkv, w = case["hq"], case["hkv"], case["window"]
    g, scale = hq // hkv, 1.0 / math.sqrt(hd)
    if case["op"] == "decode":
        out = torch.empty(len(s["lens"]), hq, hd, dtype=torch.float64, device="cuda")
        for i, n in enumerate(s["lens"]):
            pages = s["table"][i, :-(-n // page)].long()
            lo = max(0, n - w) if w else 0
            for h in range(hkv):
                k = s["kc"][pages, h].reshape(-1, hd)[lo:n].double()
                v = s["vc"][pages, h].reshape(-1, hd)[lo:n].double()
                out[i, h * g:(h + 1) * g] = torch.softmax(s["q"][i, h * g:(h + 1) * g].double() @ k.T * scale, -1) @ v
        return out
    out = torch.empty(sum(s["lens"]), hq, hd, dtype=torch.float64, device="cuda")
    t = 0
    for n in s["lens"]:
        mask = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        if w:
            mask &= torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1 - w)
        for h in range(hq):
            a = (s["q"][t:t + n, h].double() @ s["k"][t:t + n, h // g].double().T) * scale
            out[t:t + n, h] = torch.softmax(a.masked_fill_(~mask, -math.inf), -1) @ s["v"][t:t + n, h // g].double()
        t += n
    return out


def _exact_sample(s):
    x, u = s["logits"].float().cpu().numpy(), s["u"].cpu().numpy()
    temp, top_k, top_p, min_p = (s[k].cpu().numpy() for k in ("t_row", "k_row", "p_row", "m_row"))
    got = []
    for r in range(x.shape[0]):
        row = x[r].astype(np.float64)
        order = np.argsort(-row, kind="stable")
        if not temp[r] > 0:
            got.append(order[0])
            continue
        w = np.exp((row[order] - row[order[0]]) / np.float64(temp[r]))
        m = int((w >= np.float64(min_p[r])).sum())
        if top_k[r] > 0:
            m = min(m, int(top_k[r]))
        c = np.cumsum(w[:m])
        if top_p[r] < 1:
            m = 1 + int(np.searchsorted(c, np.float64(top_p[r]) * c[-1], side="left"))
        kept = np.sort(order[:m])
        c = np.cumsum(np.exp((row[kept] - row[order[0]]) / np.float64(temp[r])))
        got.append(kept[int(np.searchsorted(c, np.float64(u[r]) * c[-1], side="right"))])
    return np.asarray(got, np.int32)
