"""Plain forms in 64 bits of the calls over device-side lengths, and the bounds their
results are held to.

Attention bound, element by element, with A = sum p |v| and S = max_t |scale| sum |q k|:
the output's rounding, half a step: finfo.eps / 2 * |o|; the weights as two 16-bit
planes, 2^-16 A in bfloat16 (one plane, where a kernel says so: finfo.eps / 2 * A);
a score's float32 error: each of the D / 16 matrix steps may truncate the running sum,
2^-22 S a step, and one more for the scaling, and an exp2 within 2^-21, so a weight is
off by delta = (D / 16 + 1) 2^-22 S + 2^-21 relative to the others, which moves o by at
most 2 delta A; and one truncation a matrix step of the sums over the tokens, 2^-22 A a
step.  lse: delta, the sums' error, and a float32 rounding of its own."""
import torch

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def attention(q, k, v, seen, scale):
    """q [T, D], k and v [N, D], seen [T, N] bool, all on the CPU in 64 bits:
    (o, lse, A, S) with the empty partial (0, -inf) for rows that see nothing."""
    x = (q @ k.T) * scale
    x = torch.where(seen, x, torch.full_like(x, float("-inf")))
    lse = torch.logsumexp(x, 1) if k.shape[0] else torch.full((q.shape[0],), float("-inf"), dtype=torch.float64)
    w = torch.where(seen, (x - lse[:, None]).exp(), torch.zeros_like(x))
    s = (q.abs() @ k.abs().T * abs(scale)).amax(1) if k.shape[0] else torch.zeros(q.shape[0], dtype=torch.float64)
    return w @ v, lse, w @ v.abs(), s


def attention_bounds(o, lse, a, s, D, n, out_dtype, in_dtype, one_plane=False):
    half = lambda t: torch.finfo(t).eps / 2  # noqa: E731
    delta = ((D // 16 + 1) * 2.0 ** -22 * s + 2.0 ** -21)[:, None]
    plane = half(in_dtype) if one_plane else 2.0 ** -16
    steps = (n // 16 + 2) * 2.0 ** -22
    tiny = torch.finfo(out_dtype).tiny * torch.finfo(out_dtype).eps  # a subnormal's step
    o_tol = half(out_dtype) * o.abs() + (plane + 2 * delta + steps) * (1 + half(out_dtype)) * a + tiny
    lse_tol = delta[:, 0] + steps + 2.0 ** -23 * torch.where(torch.isinf(lse), torch.zeros_like(lse), lse.abs())
    return o_tol, lse_tol


def check_attention(got_o, got_lse, want, D, n, in_dtype, one_plane=False, what=""):
    o, lse, a, s = want
    o_tol, lse_tol = attention_bounds(o, lse, a, s, D, n, got_o.dtype, in_dtype, one_plane)
    got_o, got_lse = got_o.double().cpu(), got_lse.double().cpu()
    assert torch.equal(torch.isinf(got_lse), torch.isinf(lse)), f"{what}: empty rows differ"
    empty = torch.isinf(lse)
    assert (got_lse[empty] == float("-inf")).all() and (got_o[empty] == 0).all(), f"{what}: empty rows"
    d = (got_o - o).abs()
    assert (d <= o_tol).all(), f"{what}: o off by {(d / o_tol).max():.2f} of its bound"
    d = (got_lse - lse).abs()[~empty]
    if d.numel():
        assert (d <= lse_tol[~empty]).all(), f"{what}: lse off by {(d / lse_tol[~empty]).max():.2f} of its bound"


class Pages:
    """Requests of the given lengths in pools whose unused rows hold NaN (keys) and
    infinities (values): a stray read shows up."""

    def __init__(self, lens, H, D, dtype, seed, max_pages=None, spare=3):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.D = list(lens), H, D
        self.dtype = DTYPES[dtype]
        need = sum(-(-n // PAGE) for n in lens)
        self.slots = need + spare
        self.max_pages = max_pages or max(1, max(-(-n // PAGE) for n in lens))
        perm = torch.randperm(self.slots, generator=gen)
        self.table = torch.full((len(lens), self.max_pages), -7, dtype=torch.int32)
        self.k = torch.full((self.slots, H, PAGE, D), float("nan"), dtype=self.dtype)
        self.v = torch.full((self.slots, H, PAGE, D), float("inf"), dtype=self.dtype)
        self.keys, self.values = [], []
        at = 0
        for b, n in enumerate(lens):
            p = -(-n // PAGE)
            self.table[b, :p] = perm[at:at + p].int()
            at += p
            k = torch.randn(n, H, D, generator=gen).to(self.dtype)
            v = torch.randn(n, H, D, generator=gen).to(self.dtype)
            self.keys.append(k.double())
            self.values.append(v.double())
            for i in range(p):
                rows = slice(i * PAGE, min(n, (i + 1) * PAGE))
                c = rows.stop - rows.start
                self.k[self.table[b, i], :, :c] = k[rows].transpose(0, 1)
                self.v[self.table[b, i], :, :c] = v[rows].transpose(0, 1)
        self.gen = gen

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.gen).to(self.dtype)


def tables_model(old, new, table, free, n_free, max_tokens):
    """tpk_kv_tables_update as a stack and a loop; table (list of lists) and free are
    changed in place.  Returns (n_free, length, granted, tok_off, slot, pos, req)."""
    pages = lambda n: (n + 63) // 64  # noqa: E731
    max_pages = len(table[0])
    n = len(old)
    valid = [a >= 0 and b >= 0 for a, b in zip(old, new)]
    grow = [max(0, b - a) if ok else (max(0, b - a) if a >= 0 else 0) for a, b, ok in zip(old, new, valid)]
    end, off, fits = 0, [0], []
    for i in range(n):
        end += grow[i]
        off.append(min(end, max_tokens))
        fits.append(valid[i] and pages(old[i]) <= max_pages and pages(new[i]) <= max_pages
                    and (grow[i] == 0 or end <= max_tokens))
    stack = list(free[:n_free])
    for i in range(n):
        if fits[i]:
            stack += table[i][pages(new[i]):pages(old[i])]
    there, want, granted = len(stack), 0, []
    for i in range(n):
        need = max(0, pages(new[i]) - pages(old[i])) if fits[i] else 0
        want += need
        ok = fits[i] and (need == 0 or want <= there)
        granted.append(int(ok))
        if ok:
            for j in range(need):
                table[i][pages(old[i]) + j] = stack.pop()
    for i in range(n_free, min(len(stack), len(free))):
        free[i] = stack[i]
    slot, pos, req = [-1] * max_tokens, [0] * max_tokens, [-1] * max_tokens
    for i in range(n):
        for t in range(off[i], off[i + 1]):
            p = old[i] + t - off[i]
            pos[t], req[t] = p, i
            if granted[i]:
                slot[t] = table[i][p // 64] * 64 + p % 64
    length = [b if ok else a for a, b, ok in zip(old, new, granted)]
    return min(len(stack), len(free)), length, granted, off, slot, pos, req
