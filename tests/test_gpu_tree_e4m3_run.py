"""All operators of speculation over forked sequences together on an E4M3 cache, whose scales pass through every step:
a prompt, forked, then steps of a drafted tree each, the accepted path kept."""
import pytest
import torch

from tests import paged_reference as R
from tests import tree_reference as X

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from query_aware_sparse_append_gb300 import build
    build.build()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Path:
    """A sequence's tokens as they should be (rotated keys and values, 64 bits), and how often each was rounded to a code
    since: once when it came, once whenever its page's scale grew, once when it came to another page."""

    def __init__(self, c, rows, b):
        self.c, self.rows, self.b = c, rows, b
        self.values = torch.zeros((2, c.hkv, 0, c.d), dtype=torch.float64, device="cuda")
        self.times = torch.zeros((2, c.hkv, 0), dtype=torch.float64, device="cuda")

    def _at(self, length):
        pos = torch.arange(length, device="cuda")
        page = self.rows[self.b].long()[pos // self.c.page]
        return page, self.c.scales[page][:, :, :2].permute(2, 1, 0).clone()      # [length], [2, hkv, length]

    def copy(self, b):
        other = Path(self.c, self.rows, b)
        other.values, other.times = self.values.clone(), self.times.clone()
        return other

    def before(self, length):
        self.page, self.scale = self._at(length)

    def appended(self, new):
        old = self.values.shape[2]
        _, scale = self._at(old + new.shape[2])
        self.times = torch.cat([self.times + (scale[:, :, :old] != self.scale[:, :, :old]), torch.ones_like(new[..., 0])], 2)
        self.values = torch.cat([self.values, new], 2)

    def kept(self, tokens):
        page, scale = self._at(len(tokens))
        tokens = torch.tensor(tokens, device="cuda")
        moved = (self.page[tokens] != page) | (self.scale[:, :, tokens] != scale)
        self.times = self.times[:, :, tokens] + moved
        self.values = self.values[:, :, tokens]

    def check(self, most):
        """Each rounding to a code moves a value y by at most r |y| + a, r = 2^-4 (and 2^-20 for quotients on a border), a =
        2^-10 of its page's scale at the time, which is at most most / 448: m of them move x by ((1 + r)^m - 1) (|x| + a / r).
        Keys are rotated in fp32 before (1e-5 of values up to some tens)."""
        r, a = 2.0 ** -4 + 2.0 ** -20, 2.0 ** -10 * most * (1 + 2.0 ** -20) / 448
        for w in range(2):
            n = self.values.shape[2]
            got = self.c.wide(w, self.b, n)
            x, m = self.values[w], self.times[w][..., None]
            tol = ((1 + r) ** m - 1) * (x.abs() + a / r) + 1e-5
            off = (got - x).abs()
            assert bool((off <= tol).all()), (w, (off - tol).max().item())


@pytest.mark.parametrize("hkv,group,d,page,window,sinks", [(2, 8, 128, 16, 60, 5), (4, 1, 64, 32, None, 0), (1, 4, 64, 16, 33, 1),
                                                           (1, 8, 128, 32, None, 0)])
@pytest.mark.parametrize("form", ["rule", "whole", "cut"])
def test_speculation_over_forked_sequences(hkv, group, d, page, window, sinks, form, monkeypatch):
    from query_aware_sparse_append_gb300 import binding as qasa
    if form == "rule":
        monkeypatch.delenv("QASA_TREE_FORM", raising=False)
    else:
        monkeypatch.setenv("QASA_TREE_FORM", form)
    hq = hkv * group
    prompt, T, steps, B = 75, 13, 5, 3
    c = R.Paged("e4m3", [0] * B, hkv, d, page, seed=131, reserve=prompt + steps * T)
    cache, g = c.library(), torch.Generator(device="cpu").manual_seed(132)
    table = qasa.rotation_table(prompt + steps * T, d, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    most = 0.0

    def raw(n, b, size):
        return (torch.randn((b, n, hq + 2 * hkv, d), generator=g) * size).half().cuda()

    def stored(x, positions):                                   # [n, heads, d] -> [2, hkv, n, d]
        k = X.rotate(x[:, hq:hq + hkv], table, [positions], [0] * (d // 2), False)
        return torch.stack([k, x[:, hq + hkv:].double()]).transpose(1, 2)

    x = raw(prompt, 1, 1.0)
    first = Path(c, c.table, 0)
    first.before(0)
    qasa.kv_append_rotated(cache, c.table[:1].contiguous(), _ints([0]), x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], table,
                           status=status)
    new = stored(x[0], torch.arange(prompt, device="cuda"))
    most = max(most, new.abs().max().item())
    first.appended(new)
    rows, lens = qasa.kv_fork(cache, c.table, _ints([prompt] + [0] * (B - 1)), _ints([0] * B),
                              _ints([-1] + [int(c.table[b, prompt // page]) for b in range(1, B)]),
                              table_out=c.table.clone(), status=status)
    c.table = first.rows = rows                                 # what the references read from now on
    paths = [first] + [first.copy(b) for b in range(1, B)]
    for p in paths:
        p.check(most)
    for step in range(steps):
        x = raw(T, B, 1.5 ** step)                              # scales grow
        parents = [X.random_parents(T, g) for _ in range(B)]
        trees = [X.tree_rows(p) for p in parents]
        mask, depths = qasa.tree_masks(_ints(parents), status=status)
        old = lens.tolist()
        for b, p in enumerate(paths):
            p.before(old[b])
        q = qasa.kv_append_positioned(cache, rows, lens, x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], table,
                                      lens[:, None] + depths, q=x[:, :, :hq], status=status)
        for b, p in enumerate(paths):
            new = stored(x[b], (lens[b] + depths[b]).long())
            most = max(most, new.abs().max().item())
            p.appended(new)
            p.check(most)
        out = qasa.tree_attention(cache, q, rows, lens + T, mask, window=window, sink_tokens=sinks, status=status)
        accepted = []
        for b in range(B):                                      # against the cache as it is: its own scales and codes
            ref, weighed, size = X.attention(c, q[b], b, old[b] + T, T, trees[b][0], window, sinks)
            tol = R.attention_tolerance(ref, weighed, size, d, torch.float16)
            err = (out[b].double() - ref).abs()
            assert bool((err <= tol).all()), (step, b, (err - tol).max().item())
            best = max(range(T), key=lambda t: (trees[b][1][t], t))
            accepted.append(sorted(trees[b][0][best]))
            paths[b].before(old[b] + T)
        longest = max(map(len, accepted))
        keep = _ints([a + [-1] * (longest - len(a)) for a in accepted])
        lens = qasa.kv_keep_tokens(cache, rows, lens + T, lens, keep, keep_lens=_ints([len(a) for a in accepted]), status=status)
        for b, p in enumerate(paths):
            p.kept(list(range(old[b])) + [old[b] + a for a in accepted[b]])
            p.check(most)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert lens.tolist() == [p.values.shape[2] for p in paths]
    # the boxes are those of the codes that are left, and the page selection works on them
    boxes = cache.page_bounds.clone()
    qasa.rebuild_page_bounds(cache, rows, lens)
    for b in range(B):
        for i in range(-(-int(lens[b]) // page)):
            assert torch.equal(boxes[int(rows[b, i])], cache.page_bounds[int(rows[b, i])])
    q = torch.randn((B, hq, d), generator=g).half().cuda()
    a, _ = qasa.sparse_decode_attention(cache, q, rows, lens, rows.shape[1])
    w = qasa.window_attention(cache, q, rows, lens)
    for b in range(B):
        ref, weighed, size = R.attention(c, q[b][None], b, int(lens[b]), 1, None, 0)
        tol = R.attention_tolerance(ref, weighed, size, d, torch.float16)[0]
        assert bool(((w[b].double() - ref[0]).abs() <= tol).all())
        assert bool(((a[b].double() - ref[0]).abs() <= 2e-3 * max(1.0, weighed.max().item()) + 1e-2 * ref[0].abs()).all())
