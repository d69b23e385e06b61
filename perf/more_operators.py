"""The cases of the operators that stand around a paged cache shared by several requests:
norms of each query and key head with the rotation and the store in the same pass, decode
attention of groups of requests that share a long prefix, attention through a sliding
window whose first tokens stay visible (one token per request, and prompts), and the
upkeep of shared pages (fork, end, compaction, and the copies that these ask for).

``run`` computes a case either in its plain form (elementary torch operations in 32
bits, rounded once) or, with ``own`` set, through the package's entry points; ``exact``
gives the same outputs from the definitions in 64 bits.  Pages hold 64 tokens; a pool
is [slot][kv_heads][64][head_dim].
"""
import random

import numpy as np
import torch

own = False

PAGE = 64
DEV = "cuda"
NINF = float("-inf")


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 48 running requests: latency
        {"op": "norm", "name": "norm_step_48", "tokens": 48, "pad": 0, "H": 8, "G": 4, "D": 128, "rot": 128, "axes": 1,
         "pairs": False, "far": 131072, "weights": True, "dtype": "bf16"},
        # a long prompt of the repository's head layout, half of each head rotated in neighbouring pairs, a padded batch
        {"op": "norm", "name": "norm_prompt_7001", "tokens": 7001, "pad": 9, "H": 4, "G": 8, "D": 256, "rot": 128, "axes": 3,
         "pairs": True, "far": 3000, "weights": True, "dtype": "f16"},
        # four answers sampled from one short prompt: latency
        {"op": "shared", "name": "shared_answers_4", "groups": 1, "least": 4, "most": 4, "plo": 1900, "phi": 1900, "olo": 60,
         "ohi": 140, "empty": 0, "H": 8, "G": 4, "D": 128, "dtype": "bf16"},
        # sixty-four chats behind one long system prompt, in the repository's head layout
        {"op": "shared", "name": "shared_prompt_64", "groups": 1, "least": 64, "most": 64, "plo": 32768, "phi": 32768, "olo": 30,
         "ohi": 1500, "empty": 0, "H": 4, "G": 8, "D": 256, "dtype": "bf16"},
        # groups of all sizes, requests that stand alone and idle slots of the batch among them, an odd head group
        {"op": "shared", "name": "shared_groups_13", "groups": 13, "least": 1, "most": 24, "plo": 300, "phi": 9000, "olo": 1,
         "ohi": 2500, "empty": 4, "H": 8, "G": 5, "D": 128, "dtype": "f16"},
        # one user's next token far into a conversation: latency
        {"op": "window", "name": "window_one", "n_req": 1, "qlo": 1, "qhi": 1, "lo": 9000, "hi": 9000, "window": 1000, "sinks": 4,
         "empty": 0, "H": 8, "G": 4, "D": 128, "dtype": "bf16"},
        # a decode batch of very different lengths, idle slots among them
        {"op": "window", "name": "window_step_120", "n_req": 120, "qlo": 1, "qhi": 1, "lo": 1, "hi": 30000, "window": 4000,
         "sinks": 70, "empty": 6, "H": 4, "G": 8, "D": 256, "dtype": "bf16"},
        # prompts, some of them the next part of a longer one
        {"op": "window", "name": "window_prompts_3", "n_req": 3, "qlo": 900, "qhi": 2500, "lo": 2500, "hi": 6000, "window": 1500,
         "sinks": 4, "empty": 0, "H": 8, "G": 4, "D": 128, "dtype": "f16"},
        # a beam search step: eight beams of eight requests change parents, some are cut back
        {"op": "fork", "name": "fork_beams_64", "parents": 8, "each": 8, "beams": True, "lo": 200, "hi": 3000, "cut": 0.1,
         "gone": 0.05, "spare": 100, "layers": 2, "H": 4, "D": 256, "max_pages": 64, "dtype": "bf16"},
        # many answers sampled from each of a few long prompts, with too few free pages for some of them
        {"op": "fork", "name": "fork_samples_400", "parents": 20, "each": 20, "beams": False, "lo": 1000, "hi": 20000, "cut": 0.2,
         "gone": 0.1, "spare": 300, "layers": 8, "H": 8, "D": 128, "max_pages": 350, "dtype": "f16"},
        # a small pool tidied in steps of a few pages while requests run
        {"op": "compact", "name": "compact_step_16", "slots": 900, "n_req": 40, "free": 0.3, "budget": 16, "layers": 4, "H": 8,
         "D": 64, "max_pages": 64, "dtype": "f16"},
        # a whole pool moved together before a part of it is given back
        {"op": "compact", "name": "compact_pool", "slots": 12000, "n_req": 200, "free": 0.4, "budget": 12000, "layers": 2, "H": 4,
         "D": 256, "max_pages": 512, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["norm", "shared", "shared", "window", "window", "fork", "compact"])
    dtype = rng.choice(["bf16", "f16"])
    D = rng.choice([64, 128, 256])
    H = rng.choice([1, 2, 4, 8]) if D < 256 else rng.choice([1, 2, 4])
    if op == "norm":
        return {"op": op, "tokens": _log(rng, 1, 7000 * 128 // D), "pad": rng.choice([0, 0, 5]), "H": H, "G": rng.choice([1, 3, 4, 8]),
                "D": D, "rot": rng.choice([D, D, D // 2, 0]), "axes": rng.choice([1, 3]), "pairs": rng.random() < 0.4,
                "far": _log(rng, 100, 1000000), "weights": rng.random() < 0.8, "dtype": dtype}
    if op == "shared":
        groups = _log(rng, 1, 13)
        most = _log(rng, 1, 64 // max(1, groups // 4))
        phi = _log(rng, 20, 30000 // groups)
        return {"op": op, "groups": groups, "least": max(1, most // rng.choice([1, 4])), "most": most, "plo": max(1, phi // rng.choice([1, 10])),
                "phi": phi, "olo": 1, "ohi": _log(rng, 2, 2000), "empty": rng.choice([0, 0, 1]), "H": H, "G": rng.choice([1, 2, 5, 8]), "D": D,
                "dtype": dtype}
    if op == "window":
        prompt = rng.random() < 0.5
        n = rng.randint(1, 4) if prompt else _log(rng, 1, 120)
        qhi = _log(rng, 2, 2000) if prompt else 1
        hi = max(qhi, _log(rng, 64, 6000 if prompt else 20000))
        return {"op": op, "n_req": n, "qlo": max(1, qhi // 3), "qhi": qhi, "lo": max(1, hi // rng.choice([1, 5, 500])), "hi": hi,
                "window": rng.choice([0, 1, _log(rng, 10, 4000), _log(rng, 10, 4000), _log(rng, 100, 4000)]) if n * hi < 200000
                else _log(rng, 10, 2000), "sinks": rng.choice([0, 1, 4, 64, 130]), "empty": rng.choice([0, n // 8]), "H": H,
                "G": rng.choice([1, 2, 4, 5, 8]), "D": D, "dtype": dtype}
    layers = rng.choice([1, 2, 5])
    if op == "fork":
        return {"op": op, "parents": _log(rng, 1, 20), "each": _log(rng, 1, 20), "beams": rng.random() < 0.5, "lo": _log(rng, 1, 1000),
                "hi": _log(rng, 1000, 8000), "cut": rng.choice([0.0, 0.2]), "gone": rng.choice([0.0, 0.1]),
                "spare": rng.choice([0, 40, 400, 400]), "layers": layers, "H": H, "D": D, "max_pages": 125 + rng.randrange(40), "dtype": dtype}
    slots = _log(rng, 20, 6000)
    return {"op": op, "slots": slots, "n_req": _log(rng, 1, 200), "free": rng.choice([0.05, 0.3, 0.6]), "budget": rng.choice([8, 100, slots]),
            "layers": layers, "H": H, "D": D, "max_pages": 300 + rng.randrange(40), "dtype": dtype}


# -------------------------------------- what a case fixes by itself, on the host
def _case_rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _pages(n):
    return -(-n // PAGE)


def _groups(case):
    """(where each group's requests begin, its prefix's tokens, each request's tokens)."""
    rng = _case_rng(case)
    off, shared, lens = [0], [], []
    for _ in range(case["groups"]):
        shared.append(rng.randint(case["plo"], case["phi"]))
        for _ in range(rng.randint(case["least"], case["most"])):
            lens.append(shared[-1] + _log(rng, case["olo"], case["ohi"]))
        off.append(len(lens))
    for b in rng.sample(range(len(lens)), min(case["empty"], len(lens) - 1)):
        lens[b] = 0  # an idle slot of the batch
    return off, shared, lens


def _prompts(case):
    """(query tokens, tokens) of each request; the query tokens are its last ones."""
    rng = _case_rng(case)
    q, n = [], []
    for b in range(case["n_req"]):
        q.append(rng.randint(case["qlo"], case["qhi"]))
        n.append(0 if b < case["empty"] else max(q[-1], _log(rng, case["lo"], case["hi"])))
    both = list(zip(q, n))
    rng.shuffle(both)
    return [a for a, _ in both], [c for _, c in both]


def _family(case):
    """A batch before a fork: (each row's tokens, the rows whose pages it begins with, how
    many of these, and what it asks for: its source and how many tokens of it)."""
    rng = _case_rng(case)
    n = case["parents"] * case["each"]
    lens, base, common, source, keep = [], [], [], [], []
    for p in range(case["parents"]):
        first = p * case["each"]
        top = _log(rng, case["lo"], case["hi"])
        for e in range(case["each"]):
            if case["beams"]:  # the beams of a request share what they began with, and each has pages of its own
                lens.append(top)
                base.append(first)
                common.append(min(top // PAGE, max(0, top // PAGE - rng.randint(0, 3))) if e else 0)
                source.append(first + rng.randrange(case["each"]))
            else:  # the first row of each holds the prompt, the others nothing yet
                lens.append(top if e == 0 else 0)
                base.append(first)
                common.append(0)
                source.append(first)
    for b in range(n):
        x = rng.random()
        if x < case["gone"]:
            source[b] = -1
        keep.append(0 if source[b] < 0 else rng.randint(0, lens[source[b]]) if x > 1 - case["cut"] else lens[source[b]])
    return lens, base, common, source, keep


def _occupied(case):
    """Pages of each request in a pool with free slots all over it."""
    rng = _case_rng(case)
    live = max(1, min(case["slots"] - 1, round(case["slots"] * (1 - case["free"]))))
    pages = [0] * case["n_req"]
    for _ in range(live):
        b = rng.randrange(case["n_req"])
        if pages[b] == case["max_pages"]:
            b = min(range(case["n_req"]), key=pages.__getitem__)
        if pages[b] < case["max_pages"]:
            pages[b] += 1
    return [max(0, p * PAGE - rng.randrange(PAGE)) for p in pages]


def _visible(case, pos):
    """How many tokens the query at position pos sees."""
    w = min(pos + 1, case["window"] or pos + 1)
    return w + min(case["sinks"], pos + 1 - w)


def work(case):
    if case["op"] == "fork":
        lens, _, _, source, keep = _family(case)
        entries = sum(_pages(k) for k in keep)
        copies = min(sum(1 for k in keep if k % PAGE), case["spare"])
        return {"bytes": 8 * entries + 24 * len(lens) + copies * case["layers"] * 4 * case["H"] * PAGE * case["D"] * 2, "flops": entries}
    if case["op"] == "compact":
        lens = _occupied(case)
        used, slots = sum(_pages(n) for n in lens), case["slots"]
        moves = min(case["budget"], used * (slots - used) // slots)
        return {"bytes": 8 * used + 16 * slots + moves * case["layers"] * 4 * case["H"] * PAGE * case["D"] * 2, "flops": slots}
    H, G, D = case["H"], case["G"], case["D"]
    if case["op"] == "norm":
        t = case["tokens"]
        return {"bytes": t * ((2 * H * G + 4 * H) * D * 2 + 4 * case["axes"] + 8), "flops": t * (H * G + H) * (4 * D + 3 * case["rot"])}
    if case["op"] == "shared":
        off, shared, lens = _groups(case)
        g = [k for k in range(len(shared)) for _ in range(off[k], off[k + 1])]
        tokens = sum(max([min(shared[k], n) for n in lens[off[k]:off[k + 1]]]) for k in range(len(shared)))
        tokens += sum(max(0, n - shared[g[b]]) for b, n in enumerate(lens))
        return {"bytes": tokens * H * D * 4 + len(lens) * H * G * (4 * D + 4), "flops": 4 * sum(lens) * H * G * D}
    q, n = _prompts(case)
    # the tokens that any of the request's queries sees
    tokens = sum(0 if b == 0 else min(b, _visible(case, b - 1) + a - 1) for a, b in zip(q, n))
    pairs = sum(_visible(case, p) for a, b in zip(q, n) for p in range(max(0, b - a), b))
    return {"bytes": tokens * H * D * 4 + sum(q) * H * G * (4 * D + 4), "flops": 4 * pairs * H * G * D}


# ----------------------------------------------------------------- prepare
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _pool(gen, dtype, *shape):
    pool = torch.empty(*shape, dtype=dtype, device=DEV)
    flat = pool.view(-1)
    for i in range(0, flat.numel(), 1 << 28):  # in parts: no 32-bit copy of a whole pool
        flat[i:i + (1 << 28)] = torch.randn(flat[i:i + (1 << 28)].shape, device=DEV, generator=gen).to(dtype)
    return pool


def _place(lens, max_pages, slots, gen):
    """A page table over a random placement (unused entries -1), and the slots left over."""
    perm = torch.randperm(slots, device=DEV, generator=gen).to(torch.int32)
    pages = _i32([_pages(n) for n in lens])[:, None].long()
    at = torch.arange(max_pages, device=DEV)
    index = pages.cumsum(0) - pages + at
    return torch.where(at < pages, perm[index.clamp(max=slots - 1)], -1), perm[int(pages.sum()):]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": case}
    if own:
        import tiered_paged_kv_gb300 as tpk
        s["tpk"] = tpk
        s["code"] = tpk.BF16 if case["dtype"] == "bf16" else tpk.F16
    {"norm": _prepare_norm, "shared": _prepare_shared, "window": _prepare_window, "fork": _prepare_fork,
     "compact": _prepare_compact}[case["op"]](s, case, gen)
    return s


def _prepare_norm(s, case, gen):
    T, rot, H, G, D, dt = case["tokens"], case["rot"], case["H"], case["G"], case["D"], _dtype(case)
    # one projection's output, q, k and v side by side; heads of different sizes
    s["qkv"] = (torch.randn(T, H * G + 2 * H, D, device=DEV, generator=gen)
                * torch.exp(torch.randn(T, H * G + 2 * H, 1, device=DEV, generator=gen))).to(dt).view(T, -1)
    s["q"], s["k"], s["v"] = s["qkv"][:, :H * G * D], s["qkv"][:, H * G * D:(H * G + H) * D], s["qkv"][:, (H * G + H) * D:]
    s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(D, device=DEV, generator=gen)).to(dt) if case["weights"] else None for _ in range(2))
    s["eps"] = 1e-6
    slots = _pages(T) + 2
    s["k_pool"], s["v_pool"] = _pool(gen, dt, slots, H, PAGE, D), _pool(gen, dt, slots, H, PAGE, D)
    perm = torch.randperm(slots, device=DEV, generator=gen)
    i = torch.arange(T, device=DEV)
    s["slot_map"] = perm[i // PAGE] * PAGE + i % PAGE
    s["live"] = T - min(case["pad"], T - 1)
    s["slot_map"][s["live"]:] = -1  # padding rows of the batch
    s["q_out"] = torch.zeros(T, H * G, D, dtype=dt, device=DEV)
    start = torch.randint(0, case["far"], (1,), device=DEV, generator=gen)
    axis = np.arange(rot // 2) % case["axes"]
    if case["axes"] == 1:
        s["positions"] = (start + i)[None].to(torch.int32).contiguous()
    else:  # frames of 24 x 32 patches: time, height and width
        s["positions"] = torch.stack([start + i // 768, start + i // 32 % 24, start + i % 32]).to(torch.int32).contiguous()
    s["axis_of"] = axis.astype(np.uint8)
    s["axis_dev"] = torch.tensor(axis, dtype=torch.int64, device=DEV)
    s["inv_freq"] = torch.tensor([1e6 ** (-2.0 * j / max(1, rot)) for j in range(rot // 2)], dtype=torch.float32, device=DEV)
    if own:
        s["shape"] = s["tpk"].PagedShape(H, G, D, dtype=s["code"], kv_slots=slots)


def _prepare_shared(s, case, gen):
    H, G, D, dt = case["H"], case["G"], case["D"], _dtype(case)
    off, shared, lens = _groups(case)
    n = len(lens)
    group = [k for k in range(len(shared)) for _ in range(off[k], off[k + 1])]
    full = [p // PAGE for p in shared]  # whole pages of the prefix: one copy for the group
    max_pages = max(_pages(max(c, shared[group[b]])) for b, c in enumerate(lens))
    slots = sum(full) + sum(max(0, _pages(max(c, shared[group[b]])) - full[group[b]]) for b, c in enumerate(lens)) + 3
    head, rest = _place([f * PAGE for f in full], max_pages, slots, gen)
    g = torch.tensor(group, device=DEV)
    whole = _i32(full).long()[g][:, None]
    total = _i32([_pages(max(c, shared[group[b]])) for b, c in enumerate(lens)]).long()[:, None]
    own_pages = total - whole
    at = torch.arange(max_pages, device=DEV)
    index = (own_pages.cumsum(0) - own_pages) + at - whole
    s["table"] = torch.where(at < whole, head[g], torch.where(at < total, rest[index.clamp(0, rest.numel() - 1)], -1)).to(torch.int32)
    s["k_pool"], s["v_pool"] = _pool(gen, dt, slots, H, PAGE, D), _pool(gen, dt, slots, H, PAGE, D)
    # a prefix that ends inside a page: every request has a copy of that page's rows, as a fork leaves them
    first = torch.tensor(off[:-1], device=DEV)[g]
    open_rows = _i32([p % PAGE for p in shared]).long()[g]
    b = torch.arange(n, device=DEV)
    mine, theirs = (s["table"][r, whole[:, 0].clamp(max=max_pages - 1)].long().clamp(min=0) for r in (b, first))
    copied = (torch.arange(PAGE, device=DEV) < open_rows[:, None])[:, None, :, None]
    for pool in (s["k_pool"], s["v_pool"]):
        pool[mine] = torch.where(copied, pool[theirs], pool[mine])
    s["q"] = torch.randn(n, H * G, D, device=DEV, generator=gen).to(dt)
    s["grp_off"], s["n_shared"], s["lens"], s["group"] = _i32(off), _i32(shared), _i32(lens), g
    s["off_host"], s["shared_host"], s["lens_host"], s["group_host"] = off, shared, lens, group
    s["o"], s["lse"] = torch.zeros(n, H * G, D, dtype=dt, device=DEV), torch.zeros(n, H * G, device=DEV)
    if own:
        s["shape"] = s["tpk"].PagedShape(H, G, D, dtype=s["code"], kv_slots=slots, max_pages=max_pages)
        s["ws_bytes"] = s["tpk"].decode_shared_workspace_bytes(s["shape"], n, len(shared))
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)


def _prepare_window(s, case, gen):
    H, G, D, dt = case["H"], case["G"], case["D"], _dtype(case)
    nq, lens = _prompts(case)
    slots = sum(_pages(n) for n in lens) + 3
    max_pages = max(1, max(_pages(n) for n in lens))
    s["table"], _ = _place(lens, max_pages, slots, gen)
    s["k_pool"], s["v_pool"] = _pool(gen, dt, slots, H, PAGE, D), _pool(gen, dt, slots, H, PAGE, D)
    s["nq"], s["lens_host"], s["off"] = nq, lens, [sum(nq[:i]) for i in range(len(nq) + 1)]
    rows = sum(nq)
    s["q"] = torch.randn(rows, H * G, D, device=DEV, generator=gen).to(dt)
    s["lens"], s["q_off"] = _i32(lens), None if case["qhi"] == 1 else _i32(s["off"])
    s["o"], s["lse"] = torch.zeros(rows, H * G, D, dtype=dt, device=DEV), torch.zeros(rows, H * G, device=DEV)
    if own:
        s["shape"] = s["tpk"].PagedShape(H, G, D, dtype=s["code"], kv_slots=slots, max_pages=max_pages)
        s["ws_bytes"] = s["tpk"].window_paged_workspace_bytes(s["shape"], case["n_req"], rows)
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)


def _layers(s, case, slots, gen):
    """Both pools of every layer in one buffer: [layer][keys, values][slot][kv_heads][64][head_dim]."""
    s["pools"] = _pool(gen, _dtype(case), case["layers"], 2, slots, case["H"], PAGE, case["D"])
    if own:
        s["shape"] = s["tpk"].PagedShape(case["H"], 1, case["D"], dtype=s["code"], kv_slots=slots)
        s["k_pools"], s["v_pools"] = ([s["pools"][i, j] for i in range(case["layers"])] for j in range(2))
        s["ws_bytes"] = s["tpk"].kv_pages_workspace_bytes(slots, s["table"].shape[0])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)


def _prepare_fork(s, case, gen):
    lens, base, common, source, keep = _family(case)
    n, max_pages = len(lens), case["max_pages"]
    c = torch.tensor(common, device=DEV)[:, None]
    alone = [max(0, _pages(a) - k) for a, k in zip(lens, common)]
    slots = sum(alone) + case["spare"] + 1
    table, rest = _place([a * PAGE for a in alone], max_pages, slots, gen)
    at = torch.arange(max_pages, device=DEV)
    shifted = torch.where(at < c, -1, table.gather(1, (at - c).clamp(min=0)))
    s["table"] = torch.where(at < c, shifted[torch.tensor(base, device=DEV)], shifted).to(torch.int32).contiguous()
    held = s["table"][s["table"] >= 0].long()
    s["shares"] = (torch.bincount(held, minlength=slots) - 1).clamp(min=0).to(torch.int32)
    s["free"] = torch.full((slots,), -1, dtype=torch.int32, device=DEV)
    s["free"][:case["spare"]] = rest[:case["spare"]]
    s["n_free"], s["lens"], s["source"], s["keep"] = _i32([case["spare"]]), _i32(lens), _i32(source), _i32(keep)
    s["slots"] = slots
    for k, size in {"shares_out": slots, "n_free_out": 1, "len_out": n, "granted": n, "copy_src": n, "copy_dst": n}.items():
        s[k] = torch.zeros(size, dtype=torch.int32, device=DEV)
    s["table_out"] = torch.full_like(s["table"], -1)
    _layers(s, case, slots, gen)


def _prepare_compact(s, case, gen):
    lens, slots = _occupied(case), case["slots"]
    s["table"], rest = _place(lens, case["max_pages"], slots, gen)
    s["table"] = s["table"].to(torch.int32).contiguous()
    n_free = rest.numel()
    s["free"] = torch.full((slots,), -1, dtype=torch.int32, device=DEV)
    s["free"][:n_free] = rest
    s["n_free"], s["lens"] = _i32([n_free]), _i32(lens)
    # some pages have holders outside this batch, as a cache of prompts has
    live = torch.ones(slots, dtype=torch.bool, device=DEV)
    live[rest.long()] = False
    s["shares"] = torch.where(live, torch.randint(0, 3, (slots,), device=DEV, generator=gen), 0).to(torch.int32)
    for k, size in {"shares_out": slots, "free_out": slots, "n_free_out": 1, "copy_src": case["budget"], "copy_dst": case["budget"],
                    "n_copies": 1, "new_slot": slots}.items():
        s[k] = torch.zeros(size, dtype=torch.int32, device=DEV)
    s["free_out"][:] = -1
    s["table_out"] = torch.full_like(s["table"], -1)
    _layers(s, case, slots, gen)


# --------------------------------------------------------------------- run
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _plain_norm(s):
    c = s["case"]
    H, G, D, rot, n = c["H"], c["G"], c["D"], c["rot"], s["live"]
    # far positions: the angle in 64 bits, its sine and cosine rounded to 32
    angle = s["positions"].double()[s["axis_dev"], :n].T * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x, heads, w):
        x = x[:n].float().view(n, heads, D)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
        if w is not None:
            x = x * w.float()
        y = x.clone()
        if c["pairs"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return y.to(s["q"].dtype)

    s["q_out"][:n] = turn(s["q"], H * G, s["wq"])
    slot, row = s["slot_map"][:n] // PAGE, s["slot_map"][:n] % PAGE
    s["k_pool"][slot, :, row] = turn(s["k"], H, s["wk"])
    s["v_pool"][slot, :, row] = s["v"][:n].view(n, H, D)
    return s["q_out"], s["k_pool"], s["v_pool"]


def _own_norm(s):
    c = s["case"]
    w = s["qkv"].stride(0)
    s["tpk"].kv_norm_rope_append(s["shape"], c["tokens"], s["q"], w, s["k"], w, s["v"], w, s["wq"], s["wk"], s["eps"], s["positions"],
                                 c["axes"], s["axis_of"], s["inv_freq"], c["rot"], c["pairs"], s["slot_map"], s["q_out"],
                                 s["q_out"].stride(0), s["k_pool"], s["v_pool"], stream=torch.cuda.current_stream())
    return s["q_out"], s["k_pool"], s["v_pool"]


def _softmax(scores):
    """(weights, their sum, log of the sum); a row that sees nothing gives (0, 1, -inf)."""
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == NINF, 0.0, m)
    p = (scores - m).exp()
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total == 0, 1.0, total), (m + total.log())[..., 0]


def _rows(pool, table, tokens):
    """The rows of a pool that hold tokens [requests, tokens] of the requests of a table, in 32 bits:
    [requests][kv_heads][tokens][head_dim]."""
    page = table.long().gather(1, tokens // PAGE).clamp(min=0)
    return pool[page, :, tokens % PAGE].float().transpose(1, 2)


def _plain_shared(s):
    c = s["case"]
    H, G, D, g = c["H"], c["G"], c["D"], s["group"]
    n, groups, P = g.numel(), c["groups"], max(s["shared_host"])
    most = max(b - a for a, b in zip(s["off_host"], s["off_host"][1:]))
    first = s["grp_off"][:-1].long()
    member = torch.arange(n, device=DEV) - first[g]
    q = s["q"].float().view(n, H, G, D)
    # the prefixes, once for each group: [groups][kv_heads][members * G][prefix tokens]
    padded = q.new_zeros(groups, most, H, G, D)
    padded[g, member] = q
    padded = padded.transpose(1, 2).reshape(groups, H, most * G, D)
    at = torch.arange(P, device=DEV)
    ends = _pages(P) * PAGE
    head = at.expand(groups, P).clamp(max=s["table"].shape[1] * PAGE - 1)
    x = (padded @ _rows(s["k_pool"], s["table"][first], head).transpose(2, 3)) * D ** -0.5
    x = x.view(groups, H, most, G, P).transpose(1, 2)[g, member]  # [requests][kv_heads][G][prefix tokens]
    seen = at < torch.minimum(s["n_shared"][g], s["lens"])[:, None]
    x = torch.where(seen[:, None, None], x, NINF)
    # what each request has of its own
    longest = max(1, max(b - s["shared_host"][s["group_host"][i]] for i, b in enumerate(s["lens_host"])))
    tail = s["n_shared"][g].long()[:, None] + torch.arange(longest, device=DEV)
    mine = tail < s["lens"][:, None]
    tail = torch.where(mine, tail, 0)
    y = (q @ _rows(s["k_pool"], s["table"], tail).transpose(2, 3)) * D ** -0.5
    y = torch.where(mine[:, None, None], y, NINF)
    p, total, lse = _softmax(torch.cat([x, y], -1))
    w = p.new_zeros(groups, most, H, G, P)
    w[g, member] = p[..., :P]
    w = w.transpose(1, 2).reshape(groups, H, most * G, P) @ _rows(s["v_pool"], s["table"][first], head)
    o = w.view(groups, H, most, G, D).transpose(1, 2)[g, member] + p[..., P:] @ _rows(s["v_pool"], s["table"], tail)
    s["o"][:], s["lse"][:] = (o / total).reshape(n, H * G, D), lse.reshape(n, H * G)
    return s["o"], s["lse"]


def _own_shared(s):
    w = s["q"].stride(0)
    s["tpk"].decode_attn_shared(s["shape"], s["lens"].numel(), s["case"]["groups"], s["q"], w, s["k_pool"], s["v_pool"], s["table"], s["lens"],
                                s["grp_off"], s["n_shared"], s["o"], w, False, s["lse"], s["ws"], s["ws_bytes"],
                                stream=torch.cuda.current_stream())
    return s["o"], s["lse"]


def _plain_window(s):
    c = s["case"]
    H, G, D, n = c["H"], c["G"], c["D"], c["n_req"]
    n_tok = s["lens"].long()[:, None]
    if s["q_off"] is None:  # one token each: the window's and the first tokens alone are read
        longest = max(1, max(s["lens_host"]))
        w = min(c["window"] or longest, longest)
        sinks = min(c["sinks"], longest)
        back = n_tok - w + torch.arange(w, device=DEV)
        head = torch.arange(sinks, device=DEV).expand(n, sinks)
        tok = torch.cat([head, back], 1)
        seen = torch.cat([head < (n_tok - w).clamp(min=0), back >= 0], 1)
        tok = torch.where(seen, tok, 0)
        x = (s["q"].float().view(n, H, G, D) @ _rows(s["k_pool"], s["table"], tok).transpose(2, 3)) * D ** -0.5
        p, total, lse = _softmax(torch.where(seen[:, None, None], x, NINF))
        s["o"][:] = (p @ _rows(s["v_pool"], s["table"], tok) / total).reshape(n, H * G, D)
        s["lse"][:] = lse.reshape(n, H * G)
        return s["o"], s["lse"]
    most, longest = max(s["nq"]), max(1, max(s["lens_host"]))
    at = torch.arange(s["q"].shape[0], device=DEV)
    req = torch.searchsorted(s["q_off"][1:].contiguous(), at, right=True)
    i = at - s["q_off"][:-1].long()[req]
    q = torch.zeros(n, most, H * G, D, device=DEV)
    q[req, i] = s["q"].float()
    q = q.view(n, most, H, G, D).permute(0, 2, 3, 1, 4).reshape(n, H, G * most, D)
    tok = torch.arange(longest, device=DEV)
    tokens = torch.where(tok < n_tok, tok, 0)
    count = (s["q_off"][1:] - s["q_off"][:-1]).long()[:, None]
    pos = (n_tok - count + torch.arange(most, device=DEV))[..., None]  # [requests][query][1]
    seen = (tok <= pos) & (tok < n_tok[..., None]) & ((tok < c["sinks"]) | (tok > pos - (c["window"] or longest + most)))
    x = (q @ _rows(s["k_pool"], s["table"], tokens).transpose(2, 3)) * D ** -0.5
    p, total, lse = _softmax(torch.where(seen[:, None, None], x.view(n, H, G, most, longest), NINF))
    o = p.view(n, H, G * most, longest) @ _rows(s["v_pool"], s["table"], tokens)
    o = (o.view(n, H, G, most, D) / total).permute(0, 3, 1, 2, 4).reshape(n, most, H * G, D)
    s["o"][:], s["lse"][:] = o[req, i], lse.permute(0, 3, 1, 2).reshape(n, most, H * G)[req, i]
    return s["o"], s["lse"]


def _own_window(s):
    c, w = s["case"], s["q"].stride(0)
    s["tpk"].window_attn_paged(s["shape"], c["n_req"], s["q"].shape[0], c["window"], c["sinks"], s["q"], w, s["q_off"], s["k_pool"],
                               s["v_pool"], s["table"], s["lens"], s["o"], w, s["lse"], s["ws"], s["ws_bytes"],
                               stream=torch.cuda.current_stream())
    return s["o"], s["lse"]


def _move_pages(s):
    """The copies of every layer's keys and values."""
    there = s["copy_src"] >= 0
    src, dst = s["copy_src"][there].long(), s["copy_dst"][there].long()
    s["pools"][:, :, dst] = s["pools"][:, :, src]


def _plain_fork(s):
    table, n_len, slots = s["table"], s["lens"].long(), s["slots"]
    n, max_pages = table.shape
    b, j = torch.arange(n, device=DEV), torch.arange(max_pages, device=DEV)
    src, keep = s["source"].long(), s["keep"].long()
    keep = torch.where(src < 0, 0, keep)
    src = torch.where(src < 0, b, src)
    changed = (src != b) | (keep != n_len)
    rows = table[src]
    held = torch.where(changed[:, None] & (j < -(-n_len // PAGE)[:, None]), table, slots).long()
    kept = torch.where(changed[:, None] & (j < (keep // PAGE)[:, None]), rows, slots).long()
    one = torch.ones(1, dtype=torch.int64, device=DEV).expand(n * max_pages)
    lost = torch.zeros(slots + 1, dtype=torch.int64, device=DEV).scatter_add(0, held.view(-1), one)
    base = s["shares"].long() + 1 - lost[:slots]
    base = base + torch.zeros(slots + 1, dtype=torch.int64, device=DEV).scatter_add(0, kept.view(-1), one)[:slots]
    # pages that end inside: one of those that go on writing a page keeps it if nobody else holds it
    inside = changed & (keep % PAGE > 0)
    last = torch.where(inside, rows.gather(1, (keep // PAGE).clamp(max=max_pages - 1)[:, None])[:, 0], slots).long()
    first = torch.full((slots + 1,), n, dtype=torch.int64, device=DEV).scatter_reduce(0, last, b, "amin")
    taken = (base == 0) & (first[:slots] < n)
    final = torch.where(taken, 1, base)
    keeps = torch.cat([taken, taken.new_zeros(1)])[last] & (first[last] == b)
    freed = (final <= 0) & (lost[:slots] > 0)
    s["shares_out"][:] = torch.where(freed, 0, final - 1).to(torch.int32)
    # the stack: pages nobody holds are pushed, the highest first; then those that copy take from the top, in order
    n_free = s["n_free"].long()
    rank = freed.flip(0).cumsum(0).flip(0)
    count = rank[0]
    slot = torch.arange(slots, device=DEV)
    stack = torch.cat([s["free"].long(), s["free"].new_zeros(slots + 1).long()])
    stack = stack.scatter(0, torch.where(freed, n_free + rank - 1, stack.numel() - 1), slot)
    there = n_free + count
    asks = inside & ~keeps
    place = asks.cumsum(0)
    gets = asks & (place <= there)
    fresh = stack[torch.where(gets, there - place, 0)]
    s["n_free_out"][:] = (there - gets.sum()).to(torch.int32)
    k = torch.arange(s["free"].numel(), device=DEV)
    s["free"][:] = torch.where((k >= n_free) & (k < s["n_free_out"]), stack[:k.numel()], s["free"]).to(torch.int32)
    refused = asks & ~gets
    length = torch.where(refused, keep // PAGE * PAGE, keep)
    s["len_out"][:], s["granted"][:] = length.to(torch.int32), (~refused).to(torch.int32)
    s["copy_src"][:], s["copy_dst"][:] = torch.where(gets, last, -1).to(torch.int32), torch.where(gets, fresh, -1).to(torch.int32)
    rows = torch.where((gets & (j == (keep // PAGE)[:, None]).T).T, fresh.to(torch.int32)[:, None], rows)
    s["table_out"][:] = torch.where(j < -(-length // PAGE)[:, None], rows, s["table_out"])
    _move_pages(s)
    return (s["table_out"], s["shares_out"], s["free"], s["n_free_out"], s["len_out"], s["granted"], s["copy_src"], s["copy_dst"],
            s["pools"])


def _own_fork(s):
    tpk, st = s["tpk"], torch.cuda.current_stream()
    n, max_pages = s["table"].shape
    tpk.kv_pages_fork(n, max_pages, s["slots"], s["source"], s["lens"], s["keep"], s["table"], s["table_out"], s["shares"], s["shares_out"],
                      s["free"], s["free"].numel(), s["n_free"], s["n_free_out"], s["len_out"], s["granted"], s["copy_src"], s["copy_dst"],
                      s["ws"], s["ws_bytes"], stream=st)
    tpk.kv_pages_copy(s["shape"], s["k_pools"], s["v_pools"], n, s["copy_src"], s["copy_dst"], stream=st)
    return (s["table_out"], s["shares_out"], s["free"], s["n_free_out"], s["len_out"], s["granted"], s["copy_src"], s["copy_dst"],
            s["pools"])


def _plain_compact(s):
    slots, budget = s["case"]["slots"], s["case"]["budget"]
    slot = torch.arange(slots, device=DEV)
    k = torch.arange(s["free"].numel(), device=DEV)
    free = torch.zeros(slots + 1, dtype=torch.bool, device=DEV)
    free[torch.where(k < s["n_free"], s["free"], slots).long()] = True
    free = free[:slots]
    low = torch.where(free, free.cumsum(0) - 1, budget).clamp(max=budget)  # free slots from the bottom
    top = torch.where(free, budget, (~free).flip(0).cumsum(0).flip(0) - 1).clamp(max=budget)  # held ones from the top
    none = torch.full((budget + 1,), -1, dtype=torch.int64, device=DEV)
    dst, src = none.scatter(0, low, slot)[:budget], none.scatter(0, top, slot)[:budget]
    goes = (dst >= 0) & (dst < src)
    s["copy_src"][:], s["copy_dst"][:] = torch.where(goes, src, -1).to(torch.int32), torch.where(goes, dst, -1).to(torch.int32)
    s["n_copies"][:] = goes.sum().to(torch.int32)
    left = torch.where(goes, src, slots)
    new = torch.cat([torch.where(free, -1, slot), slot.new_zeros(1)]).scatter(0, left, dst)[:slots]
    s["new_slot"][:] = new.to(torch.int32)
    shares = torch.where(free, 0, s["shares"].long())
    s["shares_out"][:] = slot.new_zeros(slots + 1).scatter(0, torch.where(new >= 0, new, slots), shares)[:slots].to(torch.int32)
    held = torch.zeros(slots + 1, dtype=torch.bool, device=DEV)
    held[torch.where(new >= 0, new, slots)] = True
    empty = ~held[:slots]
    rank = torch.where(empty, empty.flip(0).cumsum(0).flip(0) - 1, slots)  # the highest at the bottom
    stack = torch.cat([s["free_out"].long(), slot.new_zeros(slots + 1 - s["free_out"].numel())])
    s["free_out"][:] = stack.scatter(0, rank, slot)[:s["free_out"].numel()].to(torch.int32)
    s["n_free_out"][:] = empty.sum().to(torch.int32)
    there = torch.arange(s["table"].shape[1], device=DEV) < -(-s["lens"].long() // PAGE)[:, None]
    s["table_out"][:] = torch.where(there, new[torch.where(there, s["table"], 0).long()].to(torch.int32), s["table_out"])
    _move_pages(s)
    return (s["table_out"], s["shares_out"], s["free_out"], s["n_free_out"], s["copy_src"], s["copy_dst"], s["n_copies"], s["new_slot"],
            s["pools"])


def _own_compact(s):
    tpk, st = s["tpk"], torch.cuda.current_stream()
    n, max_pages = s["table"].shape
    tpk.kv_pages_compact(n, max_pages, s["case"]["slots"], s["lens"], s["table"], s["table_out"], s["shares"], s["shares_out"], s["free"],
                         s["free_out"], s["free"].numel(), s["n_free"], s["n_free_out"], s["new_slot"], s["case"]["budget"], s["copy_src"],
                         s["copy_dst"], s["n_copies"], s["ws"], s["ws_bytes"], stream=st)
    tpk.kv_pages_copy(s["shape"], s["k_pools"], s["v_pools"], s["case"]["budget"], s["copy_src"], s["copy_dst"], stream=st)
    return (s["table_out"], s["shares_out"], s["free_out"], s["n_free_out"], s["copy_src"], s["copy_dst"], s["n_copies"], s["new_slot"],
            s["pools"])


_run_plain = {"norm": _plain_norm, "shared": _plain_shared, "window": _plain_window, "fork": _plain_fork, "compact": _plain_compact}
_run_own = {"norm": _own_norm, "shared": _own_shared, "window": _own_window, "fork": _own_fork, "compact": _own_compact}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "shared": _exact_shared, "window": _exact_window, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](s)


def _exact_norm(s):
    c = s["case"]
    n, rot, D, H = s["live"], c["rot"], c["D"], c["H"]
    pos = s["positions"].double()
    out = []
    for x, heads, w in ((s["q"], H * c["G"], s["wq"]), (s["k"], H, s["wk"])):
        x = x[:n].double().reshape(n, heads, D)
        y = x / (x.square().sum(2, keepdim=True) / D + s["eps"]).sqrt()
        if w is not None:
            y = y * w.double()
        for j in range(rot // 2):
            lo, hi = (2 * j, 2 * j + 1) if c["pairs"] else (j, j + rot // 2)
            turn = torch.polar(torch.ones_like(pos[0, :n]), pos[int(s["axis_of"][j]), :n] * float(s["inv_freq"][j]))
            z = torch.complex(y[:, :, lo], y[:, :, hi]) * turn[:, None]
            y[:, :, lo], y[:, :, hi] = z.real, z.imag
        out.append(y)
    q_out, kp, vp = s["q_out"].double(), s["k_pool"].double(), s["v_pool"].double()
    q_out[:n] = out[0]
    at = s["slot_map"][:n] // PAGE * H * PAGE + s["slot_map"][:n] % PAGE
    at = (at[:, None] + torch.arange(H, device=DEV) * PAGE).reshape(-1)
    kp.view(-1, D)[at] = out[1].reshape(-1, D)
    vp.view(-1, D)[at] = s["v"][:n].double().reshape(-1, D)
    return q_out, kp, vp


def _exact_rows(s, o, lse, rows, slot_row, tok, hide):
    """Queries `rows` over the tokens at slot_row = (slot, row in it); hide: [query][token]."""
    H, G, D = s["case"]["H"], s["case"]["G"], s["case"]["D"]
    q = s["q"][rows].double()
    bias = torch.zeros(q.shape[0], tok, dtype=torch.float64, device=DEV).masked_fill(hide, NINF)
    for h in range(H):
        k, v = (pool[slot_row[0], h, slot_row[1]].double() for pool in (s["k_pool"], s["v_pool"]))
        for j in range(h * G, h * G + G):
            logits = torch.einsum("td,nd->tn", q[:, j], k) / D ** 0.5 + bias
            total = torch.logsumexp(logits, 1) if tok else torch.full((q.shape[0],), NINF, dtype=torch.float64, device=DEV)
            lse[rows, j] = total
            o[rows, j] = torch.einsum("tn,nd->td", torch.where(hide, 0.0, (logits - total[:, None]).exp()), v)


def _exact_shared(s):
    """Each request by itself over its own table row."""
    o, lse = s["o"].double(), s["lse"].double()
    for b, n in enumerate(s["lens_host"]):
        at = torch.arange(n, device=DEV)
        page = s["table"][b].long().repeat_interleave(PAGE)[:n]
        _exact_rows(s, o, lse, slice(b, b + 1), (page, at % PAGE), n, torch.zeros(1, n, dtype=torch.bool, device=DEV))
    return o, lse


def _exact_window(s):
    c = s["case"]
    o, lse = s["o"].double(), s["lse"].double()
    for b, n in enumerate(s["lens_host"]):
        at = torch.arange(n, device=DEV)
        page = s["table"][b].long().repeat_interleave(PAGE)[:n]
        pos = torch.arange(n - s["nq"][b], n, device=DEV)[:, None]
        hide = at > pos
        if c["window"]:
            hide = hide | ((pos - at >= c["window"]) & (at >= c["sinks"]))
        _exact_rows(s, o, lse, slice(s["off"][b], s["off"][b + 1]), (page, at % PAGE), n, hide)
    return o, lse


def _exact_fork(s):
    """Holders counted one by one, and a free stack."""
    table, lens, source, keep = (s[k].tolist() for k in ("table", "lens", "source", "keep"))
    n, shares = len(lens), s["shares"].tolist()
    n_free = int(s["n_free"])
    stack = s["free"].tolist()[:n_free]
    want = [0 if p < 0 else k for p, k in zip(source, keep)]
    src = [b if p < 0 else p for b, p in enumerate(source)]
    moved = [b for b in range(n) if src[b] != b or want[b] != lens[b]]
    holders = {}
    for b in moved:
        for x in table[b][:_pages(lens[b])]:
            holders[x] = holders.get(x, shares[x] + 1) - 1
    for b in moved:
        for x in table[src[b]][:want[b] // PAGE]:
            holders[x] = holders.get(x, shares[x] + 1) + 1
    rows = [list(table[src[b]][:_pages(want[b])]) for b in range(n)]
    copies = []
    for b in moved:
        if want[b] % PAGE:
            x = rows[b][-1]
            holders.setdefault(x, shares[x] + 1)
            if holders[x] == 0:
                holders[x] = -1  # the first to write on keeps it; negative: not for those that come
            else:
                copies.append(b)
    for x in sorted(holders, reverse=True):
        if holders[x] == 0:
            stack.append(x)
        shares[x] = max(0, abs(holders[x]) - 1)
    length, granted, copy_src, copy_dst = list(want), [1] * n, [-1] * n, [-1] * n
    for b in copies:
        if stack:
            copy_src[b], copy_dst[b] = rows[b][-1], stack.pop()
            rows[b][-1] = copy_dst[b]
        else:
            granted[b], length[b] = 0, want[b] // PAGE * PAGE
            rows[b].pop()
    free = s["free"].tolist()
    free[n_free:len(stack)] = stack[n_free:]
    out = s["table_out"].tolist()
    for b in range(n):
        out[b][:len(rows[b])] = rows[b]
    pools = s["pools"].clone()
    for x, y in zip(copy_src, copy_dst):
        if x >= 0:
            pools[:, :, y] = s["pools"][:, :, x]
    i32 = lambda x: np.array(x, np.int32)  # noqa: E731
    return i32(out), i32(shares), i32(free), i32([len(stack)]), i32(length), i32(granted), i32(copy_src), i32(copy_dst), pools.double()


def _exact_compact(s):
    """The lowest free slot takes the highest page, over and over."""
    slots, budget = s["case"]["slots"], s["case"]["budget"]
    free = sorted(s["free"].tolist()[:int(s["n_free"])])
    is_free = set(free)
    held = [x for x in range(slots) if x not in is_free]
    new = [-1 if x in is_free else x for x in range(slots)]
    moves = []
    for y, x in zip(free, reversed(held)):
        if y > x or len(moves) == budget:
            break
        moves.append((x, y))
        new[x] = y
    shares, old = [0] * slots, s["shares"].tolist()
    for x in held:
        shares[new[x]] = old[x]
    used = {new[x] for x in held}
    stack = [x for x in range(slots - 1, -1, -1) if x not in used]
    out, rows = s["table_out"].tolist(), s["table"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        out[b][:_pages(n)] = [new[x] for x in rows[b][:_pages(n)]]
    pools = s["pools"].clone()
    for x, y in moves:
        pools[:, :, y] = s["pools"][:, :, x]
    i32 = lambda x: np.array(x, np.int32)  # noqa: E731
    pad = [-1] * (budget - len(moves))
    free_out = s["free_out"].tolist()
    free_out[:len(stack)] = stack
    return (i32(out), i32(shares), i32(free_out), i32([len(stack)]), i32([x for x, _ in moves] + pad), i32([y for _, y in moves] + pad),
            i32([len(moves)]), i32(new), pools.double())
