"""lora_qk_norm_rope against a 64-bit reference."""
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L

pytestmark = pytest.mark.gpu

EPS = 1e-6


class Case:
    def __init__(self, T, heads=(4, 2, 64), rot=None, interleaved=0, weights=True, slots=True, copy_v=True, pad=0,
                 max_pos=100, seed=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.T, (self.hq, self.hkv, self.d) = T, heads
        self.rot = self.d if rot is None else rot
        self.inter, self.max_pos, self.pad = interleaved, max_pos, pad
        qc, kc = self.hq * self.d, self.hkv * self.d
        self.qkv = torch.full((T, qc + 2 * kc + pad), float("nan"), dtype=torch.bfloat16)
        self.qkv[:, :qc + 2 * kc] = (spread * torch.randn(T, qc + 2 * kc, generator=g)).to(torch.bfloat16)
        self.w = [(1 + 0.3 * torch.randn(self.d, generator=g)).to(torch.bfloat16) if weights else None for _ in "qk"]
        self.pos = torch.randint(0, max_pos, (T,), generator=g, dtype=torch.int32)
        self.cs = torch.randn(max_pos, max(1, self.rot), generator=g)
        self.rows = T + 5 if slots else T
        self.slots = torch.randperm(self.rows, generator=g)[:T].to(torch.int32) if slots else None
        self.copy_v = copy_v

    def desc(self):
        return L.RopeDesc(n_q_heads=self.hq, n_kv_heads=self.hkv, head_dim=self.d, rot_dim=self.rot,
                          interleaved=self.inter, max_pos=self.max_pos, eps=EPS)

    def reference(self):
        """(values, the magnitudes their fp32 terms have) of [T][hq + 2 hkv][d]."""
        n = self.hq + 2 * self.hkv
        x = self.qkv[:, :n * self.d].double().view(self.T, n, self.d)
        y, mag = x.clone(), x.abs()
        h = self.rot // 2
        for lo, hi, w in ((0, self.hq, self.w[0]), (self.hq, self.hq + self.hkv, self.w[1])):
            z = x[:, lo:hi]
            z = z / (z.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
            if w is not None:
                z = z * w.double()
            o, m = z.clone(), z.abs()
            if h:
                cs = self.cs[self.pos.long()].double()[:, None, :]
                co, si = cs[..., :h], cs[..., h:self.rot]
                a, b = ((z[..., 0:self.rot:2], z[..., 1:self.rot:2]) if self.inter
                        else (z[..., :h], z[..., h:self.rot]))
                p, q = a * co - b * si, b * co + a * si
                mp, mq = (a * co).abs() + (b * si).abs(), (b * co).abs() + (a * si).abs()
                if self.inter:
                    o[..., 0:self.rot:2], o[..., 1:self.rot:2] = p, q
                    m[..., 0:self.rot:2], m[..., 1:self.rot:2] = mp, mq
                else:
                    o[..., :h], o[..., h:self.rot] = p, q
                    m[..., :h], m[..., h:self.rot] = mp, mq
            y[:, lo:hi], mag[:, lo:hi] = o, m
        return y, mag

    def run(self, status=None):
        self.dqkv = self.qkv.cuda()
        qc, kc = self.hq * self.d, self.hkv * self.d
        self.q = torch.full((self.T, qc + self.pad), 7.0, dtype=torch.bfloat16, device="cuda")
        self.k = torch.full((self.rows, kc + self.pad), 7.0, dtype=torch.bfloat16, device="cuda")
        self.v = torch.full((self.rows, kc + self.pad), 7.0, dtype=torch.bfloat16, device="cuda")
        w = [x.cuda() if x is not None else None for x in self.w]
        sl = self.slots.cuda() if self.slots is not None else None
        self.keep = (w, sl, self.pos.cuda(), self.cs.cuda())
        L.lora_qk_norm_rope(self.desc(), self.dqkv, self.dqkv.stride(0), self.T, w[0], w[1], self.keep[2],
                            self.keep[3], self.q, self.q.stride(0), self.k, self.k.stride(0),
                            self.v if self.copy_v else None, self.v.stride(0), sl, self.rows, status)
        torch.cuda.synchronize()
        return self

    def check(self, skipped=(), no_kv=()):
        """One rounding to bf16 (at most 2^-8 of the value) and about a dozen fp32 roundings of the terms."""
        ref, mag = self.reference()
        qc, kc = self.hq * self.d, self.hkv * self.d
        place = self.slots.long() if self.slots is not None else torch.arange(self.T)
        live = torch.tensor([t not in skipped for t in range(self.T)])
        kv = torch.tensor([t not in skipped and t not in no_kv for t in range(self.T)])

        def close(got, a, b, rows):
            n = (b - a)
            r, m = ref[rows][:, a:b].reshape(-1, n * self.d), mag[rows][:, a:b].reshape(-1, n * self.d)
            assert torch.all((got.double() - r).abs() <= 2.0 ** -8 * r.abs() + 2.0 ** -19 * m)

        q, k, v = self.q.cpu(), self.k.cpu(), self.v.cpu()
        close(q[live][:, :qc], 0, self.hq, live)
        close(k[place[kv]][:, :kc], self.hq, self.hq + self.hkv, kv)
        n = self.hq + self.hkv
        if self.copy_v:
            want = self.qkv[kv][:, n * self.d:(n + self.hkv) * self.d]
            assert torch.equal(v[place[kv]][:, :kc].contiguous().view(torch.int16), want.contiguous().view(torch.int16))
        else:
            assert torch.all(v == 7.0)
        free = torch.ones(self.rows, dtype=torch.bool)
        free[place[kv]] = False
        assert torch.all(k[free] == 7.0) and torch.all(v[free] == 7.0) and torch.all(q[~live] == 7.0)
        if self.pad:
            assert torch.all(q[:, qc:] == 7.0) and torch.all(k[:, kc:] == 7.0) and torch.all(v[:, kc:] == 7.0)


@pytest.mark.parametrize("d,rot", [(8, 8), (16, 8), (64, 64), (64, 32), (80, 80), (96, 48), (128, 128), (128, 64),
                                   (192, 64), (256, 256), (128, 0), (40, 24)])
@pytest.mark.parametrize("inter", [0, 1])
def test_head_sizes(d, rot, inter):
    Case(13, heads=(5, 2, d), rot=rot, interleaved=inter, seed=d + rot).run().check()


@pytest.mark.parametrize("heads", [(1, 1, 128), (32, 8, 128), (28, 4, 128), (16, 16, 64), (3, 1, 96), (71, 1, 64)])
@pytest.mark.parametrize("T", [1, 2, 37])
def test_head_counts(heads, T):
    Case(T, heads=heads, seed=T).run().check()


def test_many_tokens():
    Case(3001, heads=(8, 2, 128), max_pos=4000, seed=1).run().check()


@pytest.mark.parametrize("heads,rot,inter,kw", [
    ((8, 2, 128), 128, 0, dict(pad=40)), ((6, 3, 64), 32, 1, {}), ((5, 1, 40), 24, 0, {}), ((7, 1, 72), 72, 1, {}),
    ((3, 1, 256), 256, 0, {}), ((8, 2, 64), 0, 0, dict(weights=False)), ((4, 2, 96), 96, 0, dict(slots=False, copy_v=False)),
    ((2, 2, 128), 64, 0, dict(slots=False))])
def test_many_tokens_of_every_kind(heads, rot, inter, kw):
    """Enough tokens for the path over row buffers, a few of them outside the tables."""
    c = Case(4000, heads=heads, rot=rot, interleaved=inter, max_pos=500, seed=10, **kw)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    skipped, no_kv = [], []
    if rot:
        c.pos[0], c.pos[1700], c.pos[3999] = -3, 500, 1 << 30
        skipped += [0, 1700, 3999]
    if c.slots is not None:
        c.slots[5], c.slots[2500], c.slots[3998] = -1, c.rows, -2
        skipped += [2500, 3998]
        no_kv.append(5)
    c.run(status)
    for t in skipped:  # for the reference, which leaves these tokens out
        c.pos[t] = 0
    if c.slots is not None:
        c.slots[torch.tensor(skipped + no_kv, dtype=torch.long)] = 0
    c.check(skipped, no_kv)
    assert int(status) == (L.CODE["LORA_ERR_DEVICE_INDEX"] if skipped else 0)


def test_many_tokens_in_place_and_again():
    c = Case(4000, heads=(4, 2, 64), slots=False, copy_v=False, max_pos=4000, seed=11)
    qc, kc = c.hq * c.d, c.hkv * c.d
    c.run().check()
    x = c.qkv.cuda()
    w, _, pos, cs = c.keep
    L.lora_qk_norm_rope(c.desc(), x, x.stride(0), c.T, w[0], w[1], pos, cs, x, x.stride(0), x[:, qc:], x.stride(0),
                        None, 0, None, c.T, None)
    assert torch.equal(x[:, :qc], c.q) and torch.equal(x[:, qc:qc + kc], c.k)
    assert torch.equal(x[:, qc + kc:].cpu(), c.qkv[:, qc + kc:])


def test_no_slots_no_weights_no_values():
    Case(20, slots=False, weights=False, copy_v=False, seed=2).run().check()


def test_padded_rows():
    Case(20, pad=24, seed=3).run().check()


def test_in_place():
    c = Case(30, slots=False, copy_v=False, seed=4)
    qc, kc = c.hq * c.d, c.hkv * c.d
    x = c.qkv.cuda()
    w = [y.cuda() for y in c.w]
    pos, cs = c.pos.cuda(), c.cs.cuda()
    L.lora_qk_norm_rope(c.desc(), x, x.stride(0), c.T, w[0], w[1], pos, cs, x, x.stride(0), x[:, qc:], x.stride(0),
                        None, 0, None, c.T, None)
    c.run()
    assert torch.equal(x[:, :qc], c.q) and torch.equal(x[:, qc:qc + kc], c.k)
    assert torch.equal(x[:, qc + kc:].cpu(), c.qkv[:, qc + kc:])
    c.check()


def test_zero_rows_and_large_values():
    c = Case(8, seed=5, spread=1e4)
    c.qkv[3] = 0
    c.run().check()
    assert torch.all(c.q[3] == 0)


def test_what_is_not_rotated_stays_apart():
    # an infinite value makes its own head NaN or zero and no other
    c = Case(4, rot=32, seed=6)
    c.qkv[1, 40] = float("inf")
    c.run()
    q = c.q.float().cpu().view(4, c.hq, c.d)
    assert torch.isnan(q[1, 0, 40]) and torch.all(q[1, 0, :40] == 0) and torch.all(q[1, 0, 41:] == 0)
    assert torch.all(torch.isfinite(q[0])) and torch.all(torch.isfinite(q[1, 1:]))


def test_tokens_outside_the_tables():
    c = Case(12, seed=7)
    c.pos[2], c.pos[5] = -1, c.max_pos
    c.slots[7], c.slots[8], c.slots[9] = -1, c.rows, -2
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.run(status)
    c.slots[7] = c.slots[8] = c.slots[9] = 0  # for the reference, which leaves these tokens out
    c.pos[2] = c.pos[5] = 0
    c.check(skipped=(2, 5, 8, 9), no_kv=(7,))
    assert int(status) == L.CODE["LORA_ERR_DEVICE_INDEX"]
    c = Case(12, seed=8)
    status.zero_()
    c.run(status).check()
    assert int(status) == 0


def test_refusals():
    c = Case(6, seed=9).run()
    w, sl, pos, cs = c.keep
    args = [c.desc(), c.dqkv, c.dqkv.stride(0), c.T, w[0], w[1], pos, cs, c.q, c.q.stride(0), c.k, c.k.stride(0), c.v,
            c.v.stride(0), sl, c.rows, None]

    def refused(i, value):
        a = list(args)
        a[i] = value
        with pytest.raises(L.LoraError) as e:
            L.lora_qk_norm_rope(*a)
        assert e.value.code == L.CODE["LORA_ERR_INVALID_ARG"]

    for i in (1, 6, 7, 8, 10):
        refused(i, None)
    for i in (1, 4, 5, 7, 8, 10, 12):
        refused(i, args[i].data_ptr() + 8)
    for i in (2, 9, 11, 13):
        refused(i, args[i] - 8)
        refused(i, args[i] + 4)
    refused(3, -1)
    refused(15, -1)
    a = list(args)
    a[14], a[15] = None, c.T - 1
    with pytest.raises(L.LoraError):
        L.lora_qk_norm_rope(*a)
    for field, value in (("n_q_heads", 0), ("n_kv_heads", 0), ("head_dim", 12), ("head_dim", 264), ("head_dim", 0),
                         ("rot_dim", 4), ("rot_dim", 72), ("rot_dim", -8), ("interleaved", 2), ("max_pos", 0),
                         ("eps", -1.0), ("eps", float("nan")), ("eps", float("inf"))):
        d = c.desc()
        setattr(d, field, value)
        refused(0, d)
    args[3] = 0
    L.lora_qk_norm_rope(*args)  # no tokens: nothing to do
