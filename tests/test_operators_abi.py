"""Refusals of the operators around the optimiser step: every bad argument is
answered with its status before anything is launched (no GPU needed)."""
import ctypes

import pytest

import tiled_newton_schulz_amd as H
from tiled_newton_schulz_amd import shape_descriptor as sd

OK, INVALID, UNSUPPORTED, LAYOUT, OVERLAP, WORKSPACE = 0, 1, 2, 3, 4, 5
P = 1 << 30


def at(k):
    return P + (k << 24)


def ref(d):
    return None if d is None else ctypes.byref(d)


def mats(ds):
    return (H.himuon_matrix_t * len(ds))(*ds)


def mm(x=sd(10, 64, ptr=at(0)), w=None, n=None, tr=0, ends=at(5), y=sd(10, 32, ptr=at(1)), dt=H.BF16):
    w = [sd(64, 32, ptr=at(2)), sd(64, 32, ptr=at(3))] if w is None else w
    return H.lib.himuon_grouped_mm(ref(x), mats(w) if w else None, len(w) if n is None else n, tr, ends, ref(y), dt, None)


def wgrad(x=sd(10, 64, ptr=at(0)), d=sd(10, 32, ptr=at(1)), ends=at(5), g=None, n=None, dt=H.BF16, ws=None, nbytes=0):
    g = [sd(64, 32, ptr=at(2)), sd(64, 32, ptr=at(3))] if g is None else g
    return H.lib.himuon_grouped_wgrad(ref(x), ref(d), ends, mats(g) if g else None, len(g) if n is None else n, dt, ws,
                                      nbytes, None)


def test_grouped_refusals():
    assert mm(x=None) == mm(y=None) == mm(w=[]) == mm(ends=None) == mm(n=0) == mm(n=-1) == INVALID
    assert mm(dt=7) == mm(dt=H.BF16_PRECISE) == UNSUPPORTED
    assert mm(x=sd(10, 63, ptr=at(0))) == INVALID                       # inner sizes differ
    assert mm(y=sd(11, 32, ptr=at(1))) == mm(y=sd(10, 31, ptr=at(1))) == INVALID
    assert mm(tr=1) == INVALID                                          # stored N x K then
    assert mm(w=[sd(64, 32, ptr=at(2)), sd(64, 33, ptr=at(3))]) == INVALID
    assert mm(w=[sd(64, 32, ptr=at(2)), H.himuon_matrix_t(None, 64, 32, 32)]) == INVALID
    assert mm(x=sd(10, 64, ld=63, ptr=at(0))) == INVALID
    assert mm(x=sd(-1, 64, ptr=at(0))) == INVALID
    assert mm(x=sd(10, 64, ptr=at(0) + 1)) == LAYOUT
    assert mm(ends=at(5) + 2) == LAYOUT
    assert mm(y=sd(10, 32, ptr=at(0))) == OVERLAP
    assert mm(y=sd(10, 32, ptr=at(3) + 64)) == OVERLAP
    assert mm(ends=at(1)) == OVERLAP
    huge = 1 << 31
    assert mm(x=sd(huge, 64, ptr=at(0)), y=sd(huge, 32, ptr=1 << 50)) == LAYOUT
    big = (1 << 31) - 1
    assert mm(x=sd(big, 64, ptr=1 << 40), w=[sd(64, 1 << 22, ptr=at(9))], y=sd(big, 1 << 22, ptr=1 << 58)) == LAYOUT
    # no rows: nothing to do, pointers of the rows are not looked at
    assert mm(x=H.himuon_matrix_t(None, 0, 64, 64), y=H.himuon_matrix_t(None, 0, 32, 32)) == OK
    assert mm(x=H.himuon_matrix_t(None, 0, 64, 63), y=H.himuon_matrix_t(None, 0, 32, 32)) == INVALID


def test_wgrad_refusals():
    assert wgrad(x=None) == wgrad(d=None) == wgrad(g=[]) == wgrad(ends=None) == wgrad(n=0) == INVALID
    assert wgrad(dt=H.BF16_PRECISE) == UNSUPPORTED
    assert wgrad(d=sd(11, 32, ptr=at(1))) == wgrad(d=sd(10, 33, ptr=at(1))) == INVALID
    assert wgrad(g=[sd(32, 64, ptr=at(2))]) == INVALID
    assert wgrad(g=[sd(64, 32, ptr=at(2) + 1)]) == LAYOUT
    assert wgrad(g=[sd(64, 32, ptr=at(2)), sd(64, 32, ptr=at(2) + 2048)]) == OVERLAP
    assert wgrad(g=[sd(64, 32, ptr=at(0))]) == wgrad(g=[sd(64, 32, ptr=at(1))]) == wgrad(g=[sd(64, 32, ptr=at(5))]) == OVERLAP
    # many rows and a small gradient: parts of the rows in a workspace
    rows = 1 << 16
    need = ctypes.c_size_t(0)
    size = lambda x, d, n, dt=H.BF16: H.lib.himuon_grouped_wgrad_workspace(ref(x), ref(d), n, dt, ctypes.byref(need))
    x, d = sd(rows, 64, ptr=1 << 40), sd(rows, 32, ptr=1 << 41)
    assert size(x, d, 2) == OK and 0 < need.value <= 4 << 20
    assert wgrad(x=x, d=d) == wgrad(x=x, d=d, ws=at(7), nbytes=need.value - 1) == wgrad(x=x, d=d, nbytes=need.value) == WORKSPACE
    assert wgrad(x=x, d=d, ws=at(7) + 8, nbytes=need.value) == LAYOUT
    assert size(sd(10, 64), sd(10, 32), 2) == OK and need.value == 0
    assert size(sd(0, 64), sd(0, 32), 2) == OK and need.value == 0
    assert size(None, d, 2) == size(x, None, 2) == size(x, d, 0) == size(x, sd(10, 32), 2) == INVALID
    assert size(sd((1 << 31) - 1, 64), sd((1 << 31) - 1, 32), 2) == LAYOUT
    assert size(x, d, 2, H.BF16_PRECISE) == UNSUPPORTED
    # more output tiles than a launch can hold
    wide = (1 << 24) - 8
    assert wgrad(x=sd(1, wide, ptr=at(0)), d=sd(1, wide, ptr=at(9)), g=[sd(wide, wide, ptr=1 << 40)]) == LAYOUT


Z = sd(6, 100, ptr=at(0))
T = sd(6, 4, ptr=at(2))


def distill(z=Z, idx=at(1), it=H.I32, t=T, tau=1.0, norm=1, weight=None, loss=at(3), lse=at(4), dz=None, dt=H.BF16,
            ws=at(20), nb=1 << 20):
    return H.lib.himuon_distill(ref(z), idx, it, ref(t), tau, norm, weight, loss, lse, ref(dz), dt, ws, nb, None)


def distill_grad(z=Z, idx=at(1), it=H.I32, t=T, tau=1.0, lse=at(4), g=at(3), dz=sd(6, 100, ptr=at(6)), dt=H.BF16):
    return H.lib.himuon_distill_grad(ref(z), idx, it, ref(t), tau, 1, lse, g, ref(dz), dt, None)


def test_distill_refusals():
    assert distill(z=None) == distill(t=None) == distill(idx=None) == distill(loss=None) == INVALID
    for tau in (0.0, -1.0, float("inf"), float("nan"), 1e-45):
        assert distill(tau=tau) == distill_grad(tau=tau) == INVALID
    assert distill(dt=H.BF16_PRECISE) == distill(it=2) == distill_grad(it=-1) == UNSUPPORTED
    assert distill(t=sd(6, H.MAX_ENTRIES + 1, ptr=at(2))) == UNSUPPORTED
    assert distill(t=sd(5, 4, ptr=at(2))) == INVALID
    assert distill(dz=sd(6, 99, ptr=at(6))) == distill(dz=sd(5, 100, ptr=at(6))) == INVALID
    assert distill(idx=at(1) + 2) == distill(idx=at(1) + 4, it=H.I64) == distill(loss=at(3) + 1) == LAYOUT
    assert distill(z=sd(6, 100, ptr=at(0) + 1)) == LAYOUT
    assert distill(dz=sd(6, 100, ptr=at(0) + 200)) == OVERLAP          # shifted over Z
    assert distill(dz=sd(6, 100, ld=104, ptr=at(0))) == OVERLAP        # Z at another stride
    assert distill(dz=sd(6, 100, ptr=at(2))) == OVERLAP                # over the teacher's values
    assert distill(loss=at(4)) == distill(loss=at(0)) == distill(weight=at(3)) == distill(lse=at(1)) == OVERLAP
    assert distill_grad(dz=None) == distill_grad(lse=None) == distill_grad(g=None) == INVALID
    assert distill_grad(dz=sd(6, 100, ptr=at(4))) == OVERLAP
    e = lambda c: H.himuon_matrix_t(None, 0, c, c)
    assert distill(z=e(100), t=e(4), idx=None, loss=None, lse=None) == OK
    n = ctypes.c_size_t(7)
    assert H.lib.himuon_distill_workspace(None, H.BF16, 1, ctypes.byref(n)) == INVALID
    assert H.lib.himuon_distill_workspace(ref(Z), H.BF16, 1, None) == INVALID
    assert H.lib.himuon_distill_workspace(ref(Z), H.BF16_PRECISE, 1, ctypes.byref(n)) == UNSUPPORTED
    assert H.lib.himuon_distill_workspace(ref(Z), H.BF16, 1, ctypes.byref(n)) == OK


def logprobs(z=Z, tok=at(1), it=H.I64, tau=1.0, top=3, logp=at(2), ent=at(3), lse=at(4), ti=at(5), tl=at(6), dt=H.BF16,
             ws=at(20), nb=1 << 20):
    return H.lib.himuon_token_logprobs(ref(z), tok, it, tau, top, logp, ent, lse, ti, tl, dt, ws, nb, None)


def logprobs_grad(z=Z, tok=at(1), it=H.I64, tau=1.0, lse=at(4), ent=at(3), gl=at(5), gh=at(6), dz=sd(6, 100, ptr=at(7)),
                  dt=H.BF16):
    return H.lib.himuon_token_logprobs_grad(ref(z), tok, it, tau, lse, ent, gl, gh, ref(dz), dt, None)


def test_logprobs_refusals():
    assert logprobs(z=None) == logprobs(tok=None) == logprobs(top=-1) == logprobs(top=101) == INVALID
    assert logprobs(ti=None) == logprobs(tl=None) == INVALID
    assert logprobs(top=H.MAX_TOP + 1) == logprobs(dt=9) == logprobs(it=5) == UNSUPPORTED
    assert logprobs(tok=at(1) + 4) == logprobs(lse=at(4) + 2) == LAYOUT
    assert logprobs(logp=at(3)) == logprobs(lse=at(0)) == logprobs(ti=at(1)) == OVERLAP
    assert logprobs(lse=at(3) + 8) == OVERLAP
    assert logprobs(tau=0.0) == logprobs_grad(tau=float("nan")) == INVALID
    assert logprobs_grad(dz=None) == logprobs_grad(lse=None) == logprobs_grad(tok=None) == logprobs_grad(ent=None) == INVALID
    assert logprobs_grad(dz=sd(6, 100, ptr=at(5))) == OVERLAP
    e = H.himuon_matrix_t(None, 0, 100, 100)
    assert logprobs(z=e, ti=None, tl=None) == OK
    n = ctypes.c_size_t(7)
    assert H.lib.himuon_token_logprobs_workspace(ref(Z), 101, H.BF16, ctypes.byref(n)) == INVALID
    assert H.lib.himuon_token_logprobs_workspace(ref(sd(6, 1000)), 65, H.BF16, ctypes.byref(n)) == UNSUPPORTED
    assert H.lib.himuon_token_logprobs_workspace(ref(Z), 3, H.BF16, ctypes.byref(n)) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 8), torch.zeros(2, 8, 8)
    ends = torch.tensor([1, 4], dtype=torch.int32)
    for call in (lambda: H.matrices(w), lambda: H.himuon_grouped_mm(x, w, ends),
                 lambda: H.himuon_grouped_wgrad(x, x, ends),
                 lambda: H.himuon_distill(x, ends, x), lambda: H.himuon_token_logprobs(x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        H.matrices([])
    with pytest.raises(ValueError):
        H.matrices(torch.zeros(2, 8, 8, 2)[..., 0].transpose(0, 1))


def test_products_of_more_tiles_than_a_launch_holds():
    """A workgroup of 256 threads a tile of 128 x 128 or 64 x 64, and at most
    2^32 - 1 threads a launch: refused as more tiles than it can hold."""
    rows = (1 << 31) - 1 - 4096   # 16,777,183 row tiles of 128, one more for each of 40 experts
    far = [1 << 40, 1 << 45]
    w = [sd(1, 1, ptr=at(2)) for _ in range(40)]
    assert mm(x=sd(rows, 1, ptr=far[0]), w=w, y=sd(rows, 1, ptr=far[1])) == LAYOUT
    g = [sd(1, rows, ptr=far[0]), sd(1, rows, ptr=far[1])]
    assert wgrad(x=sd(1, 1, ptr=at(0)), d=sd(1, rows, ptr=1 << 50), g=g) == LAYOUT


def test_assembly_names_the_registers_it_writes():
    """Inline assembly that sets m0 says so: the compiler sets it itself, for
    instructions of its own."""
    import glob
    import os
    import re
    seen = 0
    for path in glob.glob(os.path.join(os.path.dirname(H.__file__), "csrc", "*")):
        text = open(path).read()
        for block in re.findall(r"\basm\b[^;]*?\(.*?\)\s*;", text, re.S):
            if re.search(r"s_mov_b32\s+m0\b", block):
                seen += 1
                assert '"m0"' in block.split(":")[-1], (path, block)
    assert seen > 0


def test_workspace_is_memory_of_the_operands_gpu():
    """A workspace on another device, or one whose elements share memory (less
    of it than its size), is refused before its address is used."""
    torch = pytest.importorskip("torch")
    size = lambda need: 0
    gpu0, gpu1 = torch.device("cuda:0"), torch.device("cuda:1")

    class Workspace:   # a GPU tensor's stand-in
        is_cuda = True

        def __init__(self, t, device):
            self.t, self.device = t, device

        def __getattr__(self, name):
            return getattr(self.t, name)

    whole = torch.zeros(4096, dtype=torch.uint8)
    kept, ptr, nbytes = H._scratch(size, "test", Workspace(whole, gpu0), gpu0)
    assert ptr.value == whole.data_ptr() and nbytes == 4096
    for bad in (Workspace(whole, gpu1), Workspace(torch.zeros(1, dtype=torch.uint8).expand(4096), gpu0),
                Workspace(whole[::2], gpu0), whole):
        with pytest.raises(ValueError):
            H._scratch(size, "test", bad, gpu0)


def test_described_matrices_refuse_moved_tensors():
    """Descriptors hold addresses: they are not used once a tensor has other
    memory than it was described with, and follow changes of its values."""
    torch = pytest.importorskip("torch")

    def described(tensors):
        first = tensors[0]
        arr = mats([sd(8, 4, ptr=t.data_ptr()) for t in tensors])
        return H.Matrices(arr, len(arr), (8, 4), False, first.dtype, first.device, tensors)

    stack = torch.zeros(3, 8, 4)
    for tensors in (stack, list(torch.zeros(3, 8, 4)), [torch.zeros(8, 4) for _ in range(3)]):
        m = described(tensors)
        assert H.matrices(m) is m
        tensors[1].fill_(2.0)
        assert H.matrices(m) is m
    moved = m.tensors[2]
    moved.data = torch.zeros(8, 4)
    with pytest.raises(ValueError):
        H.matrices(m)
    m = described(stack)
    stack.set_(torch.zeros(3, 8, 4))
    with pytest.raises(ValueError):
        H.matrices(m)
    m = described(stack)
    stack.untyped_storage().resize_(0)
    with pytest.raises(ValueError):
        H.matrices(m)


def test_plan_of_many_experts():
    """Experts past those of one launch are planned by their share of the rows:
    256 rows an expert are too few to cut into parts, however few experts the
    last launch holds."""
    need = ctypes.c_size_t(0)

    def size(n, rows):
        assert H.lib.himuon_grouped_wgrad_workspace(ref(sd(n * rows, 64)), ref(sd(n * rows, 64)), n, H.BF16,
                                                    ctypes.byref(need)) == OK
        return need.value

    for n in (128, 255, 256, 257, 300, 510, 511, 600):
        assert size(n, 256) == 0, n
    assert size(1, 65536) > 0


def test_temperatures_whose_exponent_factor_overflows():
    """The kernels take exponents times log2(e) / temperature: a temperature that
    leaves it infinite would make every row NaN."""
    for tau in (3.5e-39, 4.2e-39):
        assert distill(tau=tau) == distill_grad(tau=tau) == logprobs(tau=tau) == logprobs_grad(tau=tau) == INVALID


@pytest.mark.parametrize("call", ["tiled_ns", "schedule", "muon", "gram", "pair_stats"])
def test_workspace_of_the_step_has_the_memory_it_states(call, monkeypatch):
    """The step's entries refuse a workspace on another device than the matrices,
    and one with less memory than the bytes stated or than it has elements,
    before the library is called; others pass as they are."""
    torch = pytest.importorskip("torch")
    called = []

    class Library:
        def __getattr__(self, name):
            if name.endswith(("_workspace", "_workspace_size")):
                return lambda *a: 0
            return lambda *a: called.append(name) or 0

    monkeypatch.setattr(H, "lib", Library())
    m = [torch.zeros(8, 8)]
    run = {"tiled_ns": lambda **k: H.himuon_tiled_ns(m, 8, 1, stream=1, **k),
           "schedule": lambda **k: H.himuon_tiled_ns_schedule(m, [8], stream=1, **k),
           "muon": lambda **k: H.himuon_muon_step(m, m, m, 8, 1, stream=1, **k),
           "gram": lambda **k: H.himuon_gram_ns(m, 1, stream=1, **k),
           "pair_stats": lambda **k: H.himuon_pair_stats(m, m, stream=1, **k)}[call]
    ws = torch.zeros(4096, dtype=torch.uint8)
    for good in (ws, ws[256:], ws[::2], ws[:0]):
        run(workspace=good)
    assert len(called) == 4
    bad = [dict(workspace=ws[:1].expand(8192)), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="meta"))]
    if call != "pair_stats":
        bad += [dict(workspace=ws, workspace_bytes=4097), dict(workspace=ws[256:], workspace_bytes=4096)]
    for k in bad:
        with pytest.raises(ValueError):
            run(**k)
    assert len(called) == 4
