"""The 8-bit AdamW entry points' argument checks, which all run before any HIP
call (the addresses below are never dereferenced), and RankStep's choices."""
import ctypes

import pytest
import torch

HP = (1e-3, 0.9, 0.999, 1e-8, 0.01)


@pytest.fixture(scope="module")
def zm():
    import zero_partitioned_mixed_partition_amd as m
    return m


def _arrays(n=1000):
    """Disjoint addresses: master, m, m scales, v, v scales, grad, param."""
    return [0x1000000 * (k + 1) for k in range(7)]


def _flat(zm, a, n=1000, first=0, step=1, h=HP, seed=0):
    return zm._binding._adamw8(*[ctypes.c_void_p(x) for x in a], n, first, step, *h, seed, None, None)


def test_flat_step_refusals(zm):
    E, R = zm._binding.ZERO_EINVAL, zm._binding.ZERO_ERANGE
    a = _arrays()
    assert _flat(zm, a, n=0) == zm._binding.ZERO_OK
    assert _flat(zm, [None] * 7, n=0) == zm._binding.ZERO_OK
    assert _flat(zm, a, n=-1) == E and _flat(zm, a, step=0) == E
    for bad in ((-1.0, 0.9, 0.999, 1e-8, 0.0), (1e-3, 1.0, 0.999, 1e-8, 0.0), (1e-3, 0.9, -0.1, 1e-8, 0.0),
                (1e-3, 0.9, 0.999, 0.0, 0.0), (float("nan"), 0.9, 0.999, 1e-8, 0.0),
                (1e-3, 0.9, 0.999, 1e-8, float("inf"))):
        assert _flat(zm, a, h=bad) == E, bad
    for first in (-128, 1, 127, 129):
        assert _flat(zm, a, first=first) == E
        assert "multiple of 128" in zm.zero_last_error()
    assert _flat(zm, a, first=(1 << 63) - 128, n=1000) == R
    assert _flat(zm, a, n=(1 << 62)) in (E, R)           # the arrays would overlap or not fit one dispatch
    for k in range(7):
        b = list(a)
        b[k] = None
        assert _flat(zm, b) == E and "NULL" in zm.zero_last_error()


@pytest.mark.parametrize("i,j,delta,clash", [
    (0, 1, 3999, True), (0, 1, 4000, False), (0, 6, 0, True), (1, 2, 999, True), (1, 2, 1000, False),
    (2, 3, 7, True), (2, 3, 8, False), (4, 5, 7, True), (3, 4, 999, True), (6, 5, 1999, True), (5, 6, 1999, True)])
def test_overlaps_are_named(zm, i, j, delta, clash):
    """Array j placed delta bytes after array i: 1,000 elements, 8 scale bytes."""
    a = _arrays()
    a[j] = a[i] + delta
    names = ("master", "exp_avg", "exp_avg_scale", "exp_avg_sq", "exp_avg_sq_scale", "grad", "param_out")
    if clash:
        assert _flat(zm, a) == zm._binding.ZERO_EINVAL
        text = zm.zero_last_error()
        assert "overlaps" in text and names[i] in text and names[j] in text, text
    else:                                               # gets past the overlap check: the list refuses a later array
        t = _table(zm, [a, [None] + _arrays()[1:]], [1000, 1000])
        assert t == zm._binding.ZERO_EINVAL and "of tensor 1" in zm.zero_last_error()


def _table(zm, rows, numels, first=0, n_tensors=None, null_list=None, out=True):
    T = len(rows)
    lists = [(ctypes.c_void_p * max(T, 1))(*[r[k] for r in rows]) for k in range(7)]
    if null_list is not None:
        lists[null_list] = None
    ns = (ctypes.c_int64 * max(T, 1))(*numels)
    h = ctypes.c_void_p()
    count = T if n_tensors is None else n_tensors
    listed = zm._binding._mt_adamw8(*lists, ns, count, first, 1, *HP, 0, None, None) if out else None
    text = zm.zero_last_error()
    st = zm._binding._mt8_create(*lists, ns, count, first, ctypes.byref(h) if out else None)
    if out:                                             # the list form makes the same checks
        assert listed == st and text.split(": ")[1:] == zm.zero_last_error().split(": ")[1:]
    if st == zm._binding.ZERO_OK:
        assert zm._binding._mt8_blocks(h) == 0
        assert zm._binding._mt8_step(h, 1, *HP, 0, None, None) == zm._binding.ZERO_OK     # nothing to do
        zm._binding._mt8_free(h)
    return st


def test_table_refusals(zm):
    E, R = zm._binding.ZERO_EINVAL, zm._binding.ZERO_ERANGE
    a, far = _arrays(), [x + 0x100000000 for x in _arrays()]
    assert _table(zm, [], []) == zm._binding.ZERO_OK
    assert _table(zm, [[None] * 7], [0]) == zm._binding.ZERO_OK
    assert _table(zm, [a], [10], out=False) == E
    assert _table(zm, [a], [10], n_tensors=-1) == E
    for k in range(7):
        assert _table(zm, [a], [10], null_list=k) == E
    assert _table(zm, [a, far], [10, -1]) == E and "tensor 1" in zm.zero_last_error()
    assert _table(zm, [a], [10], first=5) == E
    assert _table(zm, [a], [1 << 50]) == R
    assert _table(zm, [a, far], [1000, 1000], first=(1 << 63) - 1024) == R
    far[1] = far[0]
    assert _table(zm, [a, far], [1000, 1000]) == E and "overlaps" in zm.zero_last_error()
    # past one launch of the list form (the table takes several): refused before any launch
    big = [0x100000000000 * (k + 1) for k in range(7)]
    lists = [(ctypes.c_void_p * 2)(big[k], a[k]) for k in range(7)]
    ns = (ctypes.c_int64 * 2)(512 * (1 << 25), 10)
    assert zm._binding._mt_adamw8(*lists, ns, 2, 0, 1, *HP, 0, None, None) == R
    assert "too large for one launch" in zm.zero_last_error()
    none = [None] * 8
    assert zm._binding._mt_adamw8(*none, 0, 0, 0, *HP, 0, None, None) == E          # step < 1
    assert zm._binding._mt_adamw8(*none, 0, 0, 1, *HP, 0, None, None) == zm._binding.ZERO_OK
    assert zm._binding._mt8_blocks(None) == -1
    assert zm._binding._mt8_step(None, 1, *HP, 0, None, None) == E
    assert zm._binding._mt8_step_sched(None, None, 0, None, None) == E
    assert zm._binding._adamw8_sched(*[None] * 7, 0, 0, None, 0, None, None) == E
    zm._binding._mt8_free(None)


def test_reduce_refusals(zm):
    E, OK = zm._binding.ZERO_EINVAL, zm._binding.ZERO_OK
    plan = zm.zero_partition_plan([4000], 2, 1)                   # S = 2000
    reps = (ctypes.c_void_p * 2)(0x100000000, 0x200000000)

    def call(rank=1, n_rep=2, begin=0, count=4000, a=None, grad=None, first=0, step=1, replicas=reps, p=plan.handle):
        a = _arrays() if a is None else a
        return zm._binding._reduce_adamw8(p, rank, replicas, n_rep, begin, count, *[ctypes.c_void_p(x) for x in a[:5]],
                                          ctypes.c_void_p(a[6]), grad, first, step, *HP, 0, None, None)

    assert call(begin=0, count=2000) == OK                       # misses rank 1's shard: nothing to do
    for bad in (dict(rank=2), dict(rank=-1), dict(n_rep=0), dict(n_rep=65), dict(begin=-1), dict(count=4001),
                dict(first=64), dict(step=0), dict(p=None), dict(replicas=None)):
        assert call(**bad) == E, bad
    for begin, count in ((2001, 1999), (2000, 100), (2128, 129), (1000, 1001)):
        assert call(begin=begin, count=count) == E, (begin, count)
        assert "multiples of 128" in zm.zero_last_error()
    for k in (0, 1, 2, 3, 4, 6):
        a = _arrays()
        a[k] = None
        assert call(a=a) == E and "NULL" in zm.zero_last_error()
    assert call(replicas=(ctypes.c_void_p * 2)(0x100000000, None)) == E and "NULL replica" in zm.zero_last_error()
    assert call(replicas=(ctypes.c_void_p * 2)(None, 0x100000000)) == E and "NULL replica" in zm.zero_last_error()
    a = _arrays()
    a[6] = 0x100000000 + 4000                                    # replica 0's slice starts 2,000 elements in
    assert call(a=a) == E and "overlaps replica 0" in zm.zero_last_error()
    assert call(grad=0x200000000 + 7998) == E and "shard_grad overlaps replica 1" in zm.zero_last_error()
    assert zm._binding._reduce_adamw8_sched(plan.handle, 0, reps, 2, 0, 4000, *[None] * 7, 0, None, 0, None, None) == E


def test_conversion_refusals(zm):
    E, OK = zm._binding.ZERO_EINVAL, zm._binding.ZERO_OK
    q, d = zm._binding._quantize8, zm._binding._dequantize8
    x, c, s = 0x1000000, 0x2000000, 0x3000000
    assert q(None, 0, 0, None, None, None) == OK and d(None, None, 0, None, None) == OK
    assert q(x, -1, 0, c, s, None) == E and d(c, s, -1, x, None) == E
    for bad in ((None, c, s), (x, None, s), (x, c, None)):
        assert q(bad[0], 10, 0, bad[1], bad[2], None) == E and d(bad[1], bad[2], 10, bad[0], None) == E
    for xx, cc, ss in ((x, x + 3999, s), (x, c, x), (x, c, c + 999)):
        assert q(xx, 1000, 0, cc, ss, None) == E and "overlaps" in zm.zero_last_error()
    assert d(x + 3999, s, 1000, x, None) == E and d(c, x - 7, 1000, x, None) == E


def test_binding_refuses_short_and_mistyped_tensors(zm):
    """The binding sees sizes that the C ABI cannot (CPU tensors: the device check comes after)."""
    f, b, h = (lambda n, t=t: torch.zeros(n, dtype=t) for t in (torch.float32, torch.uint8, torch.int16))
    hyper = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    good = [f(300), b(300), b(3), b(300), b(3), h(300), h(300)]
    for k in range(1, 7):
        bad = list(good)
        bad[k] = bad[k][:-1]
        with pytest.raises(ValueError, match="elements"):
            zm.zero_shard_adamw8_step(*bad, 1, **hyper)
        with pytest.raises(ValueError, match="elements"):
            zm.MultiTensor8Table(*[[x] for x in bad])
    with pytest.raises(ValueError, match="device tensor"):
        zm.zero_shard_adamw8_step(*good, 1, **hyper)
    with pytest.raises(ValueError, match="same length"):
        zm.MultiTensor8Table(*[[x] for x in good[:6]], [])
    with pytest.raises(ValueError):
        zm.zero_state8_quantize(f(300), b(299), b(3))
    with pytest.raises(ValueError):
        zm.zero_state8_dequantize(b(300), b(2), f(300))
    plan = zm.zero_partition_plan([300], 1, 1)
    with pytest.raises(ValueError):
        zm.zero_reduce_adamw8_step(plan, 0, [h(299)], 0, 300, *good[:5], good[6], 1, **hyper)
    with pytest.raises(ValueError):
        zm.zero_reduce_adamw8_step(plan, 0, [h(300)], 0, 300, *good[:4], b(2), good[6], 1, **hyper)
    assert zm.state8_blocks(0) == 0 and zm.state8_blocks(1) == 1 and zm.state8_blocks(129) == 2


def test_rank_step_options(zm):
    from zero_partitioned_mixed_partition_amd import step
    plan = zm.zero_partition_plan([5000], 4, 128)                 # S = 1280
    with pytest.raises(ValueError, match="state_bits"):
        step.RankStep(plan, 0, 1, step.Hyper(), 1.0, torch.device("cpu"), state_bits=16)
    with pytest.raises(ValueError, match="fp32 moments"):
        step.RankStep(plan, 0, 1, step.Hyper(), 1.0, torch.device("cpu"), state_bits=8, offload=True)
    rs = step.RankStep(plan, 3, 1, step.Hyper(), 0.0, torch.device("cpu"), state_bits=8)
    assert rs.exp_avg.dtype == torch.uint8 and rs.exp_avg_scale.numel() == 10 and rs.first_element == 3 * 1280
    assert rs._whole_blocks([(0, 5120, [])]) and rs._whole_blocks([(3840, 128, []), (3968, 1152, [])])
    assert not rs._whole_blocks([(3841, 1279, [])]) and not rs._whole_blocks([(3840, 100, [])])
    assert rs._whole_blocks([(0, 100, [])])                       # misses the shard
    called = []
    rs.reduce_update = lambda w, st=None: called.append("one pass")
    rs.reduce = lambda w, st=None: called.append("reduce")
    rs.clip = rs.adamw = rs.gather = lambda st=None: None
    rs.step([(0, 5120, [None])])
    rs.step([(3841, 1279, [None])])
    assert called == ["one pass", "reduce"]
    thirty_two = step.RankStep(plan, 3, 1, step.Hyper(), 0.0, torch.device("cpu"))
    assert thirty_two._whole_blocks([(3841, 1, [])])
    with pytest.raises(ValueError, match="8 bits"):
        thirty_two.moments()
    per = step.RankStep(plan, 1, 1, step.Hyper(), 0.0, torch.device("cpu"), state_bits=8, per_param=True)
    assert per.first_element == 128 * 11 and per.exp_avg_scale_tensors[0].numel() == 10


class _Stand:
    """What the binding asks of a device tensor; the address is never dereferenced."""

    def __init__(self, n, size, device, address):
        self.n, self.size, self.dev, self.address = n, size, device, address
        self.is_cuda = True
        self.device = torch.device("cuda", device)

    def numel(self):
        return self.n

    def element_size(self):
        return self.size

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return self.address


def _stands(devices):
    sizes = (4, 1, 1, 1, 1, 2, 2)
    return [_Stand(3 if k in (2, 4) else 300, size, dev, 0x1000000 * (k + 1))
            for k, (size, dev) in enumerate(zip(sizes, devices))]


def test_tensors_of_another_device_are_refused(zm, monkeypatch):
    """The default stream's handle is the same on every device: a call for another device's tensors, or one that
    mixes devices, would run on the current one with their addresses."""
    hyper = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    plan = zm.zero_partition_plan([300], 1, 1)
    cases = [([1] * 7, "the current device is 0")]
    for k in range(1, 7):
        cases.append(([int(j == k) for j in range(7)], "the call runs on device 0"))
    for devices, text in cases:
        t = _stands(devices)
        with pytest.raises(ValueError, match=text):
            zm.zero_shard_adamw8_step(*t, 1, stream=0, **hyper)
        with pytest.raises(ValueError, match=text):
            zm.MultiTensor8Table(*[[x] for x in t])
        with pytest.raises(ValueError, match=text):
            zm.zero_multi_tensor_adamw8_step(*[[x] for x in t], 1, stream=0, **hyper)
        with pytest.raises(ValueError, match=text):
            zm.zero_reduce_adamw8_step(plan, 0, [t[5]], 0, 300, *t[:5], t[6], 1, stream=0, **hyper)
    here = _stands([0] * 7)
    far = _Stand(300, 4, 1, 0x9000000)
    with pytest.raises(ValueError, match="clip_scale lies on device 1"):
        zm.zero_shard_adamw8_step(*here, 1, clip_scale=far, stream=0, **hyper)
    with pytest.raises(ValueError, match="clip_scale lies on device 1"):
        zm.zero_multi_tensor_adamw8_step(*[[x] for x in here], 1, clip_scale=far, stream=0, **hyper)
    with pytest.raises(ValueError, match="shard_grad lies on device 1"):
        zm.zero_reduce_adamw8_step(plan, 0, [here[5]], 0, 300, *here[:5], here[6], 1, stream=0,
                                   shard_grad=_Stand(300, 2, 1, 0x9000000), **hyper)
    with pytest.raises(ValueError, match="the current device is 0"):
        zm.zero_state8_quantize(far, here[1], here[2])
    with pytest.raises(ValueError, match="scales lies on device 1"):
        zm.zero_state8_quantize(here[0], here[1], _Stand(3, 1, 1, 0x9000000))
    with pytest.raises(ValueError, match="the current device is 0"):
        zm.zero_state8_dequantize(here[1], here[2], far)
    with pytest.raises(ValueError, match="codes lies on device 1"):
        zm.zero_state8_dequantize(_Stand(300, 1, 1, 0x9000000), here[2], here[0])
