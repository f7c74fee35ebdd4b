"""Host-side checks of the operators around slikl_grad: every refusal comes from the host's own
checks, before a CUDA call (so they run without a GPU, with pointers that nothing follows), the
binding's refusals, and the struct layouts against a C99 caller."""

import ctypes
import importlib.metadata
import os
import shutil
import subprocess
import sys

import pytest
import torch

import sparse_lightning_indexer_b200 as sli
from sparse_lightning_indexer_b200 import build as slibuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULLPTR, INVALID = sli.SLIKL_ERR_PARAM_NULLPTR, sli.SLIKL_ERR_PARAM_INVALID


@pytest.fixture(scope="module")
def lib():
    slibuild.build()
    return sli.load_library()


def side(T=32, S=16, N=8, x_stride=0, dx_stride=0, norm=sli.SLIKL_NORM_RMS, reserved=0):
    return sli.slikl_qk_side(T, S, N, x_stride, dx_stride, norm, reserved)


def qk_problem():
    return sli.slikl_qk_problem(sli.SLIKL_BF16, sli.SLIKL_ROT_HALVES, 128, 64, 1000, 1e-6, 0, side(),
                                side(N=1, norm=sli.SLIKL_NORM_LAYER))


def qk_tensors(gradient=False):
    tn = sli.slikl_qk_tensors()
    at = 0x10000
    for s in (tn.q, tn.k):
        for n in ("x", "gain", "positions") + (("dy", "dx", "dgain") if gradient else ("y", "keep8", "keep8_scale")):
            setattr(s, n, at)
            at += 0x10000
    tn.k.bias = 0x900000
    if gradient:
        tn.k.dbias = 0x910000
    tn.cos_sin = 0x920000
    return tn


def put(pr, path, value):
    at = pr
    *way, last = path.split(".")
    for w in way:
        at = getattr(at, w)
    setattr(at, last, value)


WS = ctypes.c_void_p(1 << 30)


def passes(call, *args, **kw):
    """Whether the call gets past every check of its arguments. The pointers here lead nowhere, so it
    is made only where there is no GPU that would follow them."""
    return torch.cuda.is_available() or call(*args, **kw) == sli.SLIKL_ERR_CUDA


def copied(struct):
    return type(struct).from_buffer_copy(struct)


def forward_rc(lib, pr, tn):
    return lib.slikl_qk_norm_rope(ctypes.byref(pr), ctypes.byref(tn), None)


def gradient_rc(lib, pr, tn, ws=WS, n=1 << 40):
    return lib.slikl_qk_norm_rope_grad(ctypes.byref(pr), ctypes.byref(tn), ws, n, None)


PROBLEM = [
    ("dtype", 2), ("rot_layout", 2), ("rot_layout", -1), ("D", 96), ("D", 256), ("D", 0), ("rot_dim", 8),
    ("rot_dim", 144), ("rot_dim", -16), ("table_rows", 0), ("table_rows", 1 << 31), ("eps", 0.0), ("eps", -1.0),
    ("eps", float("nan")), ("eps", float("inf")), ("reserved", 1), ("q.T", -1), ("q.T", 1 << 31), ("q.T", 1 << 28),
    ("q.N", 0), ("q.N", 129), ("k.norm", 3), ("k.norm", -1), ("q.reserved", 1), ("q.x_stride", 8 * 128 - 8),
    ("q.x_stride", 8 * 128 + 4), ("q.x_stride", -1024), ("k.dx_stride", 120), ("k.x_stride", 1 << 31),
]


@pytest.mark.parametrize("path,value", PROBLEM)
def test_problem_refused(lib, path, value):
    pr = qk_problem()
    put(pr, path, value)
    assert forward_rc(lib, pr, qk_tensors()) == INVALID
    assert gradient_rc(lib, pr, qk_tensors(True)) == INVALID
    n = ctypes.c_size_t(0)
    assert lib.slikl_qk_norm_rope_grad_workspace_size(ctypes.byref(pr), ctypes.byref(n)) == INVALID


@pytest.mark.parametrize("path,value,rc,gradient", [
    ("q.x", None, NULLPTR, None), ("q.y", None, None, False), ("k.keep8_scale", None, NULLPTR, False),
    ("k.keep8", None, NULLPTR, False), ("cos_sin", None, NULLPTR, None), ("cos_sin", 0x920004, INVALID, None),
    ("q.x", 0x10008, INVALID, None), ("q.y", 0x10002, INVALID, False), ("q.keep8", 0x10008, INVALID, False),
    ("q.keep8_scale", 0x10002, INVALID, False), ("q.gain", 0x10004, INVALID, None), ("k.bias", 0x10008, INVALID, None),
    ("q.bias", 0x10000, INVALID, None), ("q.positions", 0x10002, INVALID, None), ("status", 0x10002, INVALID, None),
    ("q.dy", None, NULLPTR, True), ("q.dx", None, NULLPTR, True), ("k.dx", 0x10008, INVALID, True),
    ("q.dbias", 0x10000, INVALID, True), ("q.dgain", 0x10002, INVALID, True),
])
def test_tensors_refused(lib, path, value, rc, gradient):
    pr = qk_problem()
    for grad, call in ((False, forward_rc), (True, gradient_rc)):
        if gradient is not None and grad != gradient:
            continue
        tn = qk_tensors(grad)
        put(tn, path, value)
        if rc is None:                        # y is not needed beside a checkpoint
            assert passes(call, lib, pr, tn)
            put(tn, path.split(".")[0] + ".keep8", None)
            put(tn, path.split(".")[0] + ".keep8_scale", None)
            assert call(lib, pr, tn) == NULLPTR
        else:
            assert call(lib, pr, tn) == rc


def test_combinations_refused(lib):
    pr, tn = qk_problem(), qk_tensors()
    tn.q.x, tn.q.x8, tn.q.x8_scale = None, 0x10000, 0x20000
    assert forward_rc(lib, pr, tn) == INVALID            # a checkpoint is written from x alone
    tn.q.keep8 = tn.q.keep8_scale = None
    assert passes(forward_rc, lib, pr, tn)
    tn.q.x8_scale = None
    assert forward_rc(lib, pr, tn) == NULLPTR
    pr, tn = qk_problem(), qk_tensors()
    pr.q.norm = sli.SLIKL_NORM_NONE                      # a gain without a norm
    assert forward_rc(lib, pr, tn) == INVALID
    pr, tn = qk_problem(), qk_tensors()
    pr.q.S, tn.q.positions = 0, None                     # neither positions nor a batch length
    assert forward_rc(lib, pr, tn) == INVALID
    pr.rot_dim = 0
    assert passes(forward_rc, lib, pr, tn)
    assert lib.slikl_qk_norm_rope(None, ctypes.byref(tn), None) == NULLPTR
    assert lib.slikl_qk_norm_rope(ctypes.byref(pr), None, None) == NULLPTR
    assert lib.slikl_qk_norm_rope_grad_workspace_size(ctypes.byref(pr), None) == sli.SLIKL_ERR_INNER_NULLPTR


def test_gradient_workspace(lib):
    pr, tn = qk_problem(), qk_tensors(True)
    n = sli.slikl_qk_norm_rope_grad_workspace_size(pr)
    assert gradient_rc(lib, pr, tn, None, n) == NULLPTR
    assert gradient_rc(lib, pr, tn, ctypes.c_void_p((1 << 30) + 128), n) == INVALID
    assert gradient_rc(lib, pr, tn, WS, n - 1) == sli.SLIKL_ERR_WORKSPACE_TOO_SMALL


def grad_problem(**kw):
    pr = sli.slikl_problem(sli.SLIKL_BF16, sli.SLIKL_BSND, sli.SLIKL_BSND, 0, 2, 16, 16, 0, 0, 8, 128, 64)
    for k, v in kw.items():
        setattr(pr, k, v)
    return pr


@pytest.mark.parametrize("path,value", [("dtype", sli.SLIKL_FP16), ("D", 64), ("q.T", 31), ("q.N", 4), ("k.T", 31),
                                        ("k.N", 2)])
def test_projected_needs_matching_problems(lib, path, value):
    n = ctypes.c_size_t(0)
    size = lib.slikl_grad_projected_workspace_size
    pr, qk = grad_problem(), qk_problem()
    assert size(ctypes.byref(pr), ctypes.byref(qk), None, ctypes.byref(n)) == 0 and n.value > 0
    put(qk, path, value)
    assert size(ctypes.byref(pr), ctypes.byref(qk), None, ctypes.byref(n)) == INVALID


def test_projected_tensors_refused(lib):
    pr, qk, qt = grad_problem(), qk_problem(), qk_tensors(True)
    need = sli.slikl_grad_projected_workspace_size(pr, qk)
    tn = sli.slikl_tensors()
    for i, name in enumerate(("w", "attn_softmax_l1norm", "sparse_indices", "dw", "softmax_out")):
        setattr(tn, name, 0x100000 * (i + 1))

    def rc(tn=tn, qt=qt, ws=WS, n=need, opt=None):
        return lib.slikl_grad_projected(ctypes.byref(pr), ctypes.byref(qk), ctypes.byref(tn), ctypes.byref(qt), ws,
                                        n, None, opt)

    assert passes(rc)
    assert rc(n=need - 1) == sli.SLIKL_ERR_WORKSPACE_TOO_SMALL
    assert rc(ws=None) == NULLPTR
    assert rc(ws=ctypes.c_void_p((1 << 30) + 8)) == INVALID
    for name in ("w", "attn_softmax_l1norm", "sparse_indices", "dw", "softmax_out"):
        t = copied(tn)
        setattr(t, name, None)
        assert rc(tn=t) == NULLPTR, name
    for name in ("x", "dx"):
        t = qk_tensors(True)
        setattr(t.k, name, None)
        assert rc(qt=t) == NULLPTR, name
    assert rc(opt=ctypes.byref(sli.make_options(7))) == INVALID
    assert rc(opt=ctypes.byref(sli.make_options(loss=0x1002))) == INVALID


def weights_tensors():
    return sli.slikl_key_weights_tensors(0x10000, 0x20000, None, None, 0x30000, 0x40000, 0x50000)


def weights_rc(lib, pr, tn, decay=1.0, ws=WS, n=1 << 40, opt=None):
    return lib.slikl_key_weights(ctypes.byref(pr), ctypes.byref(tn), decay, ws, n, None, opt)


@pytest.mark.parametrize("field,value", [("B", 0), ("S1", 0), ("S2", 0), ("topk", 0), ("topk", 8193), ("layout_q", 2),
                                         ("layout_k", 5), ("S1", 1 << 30)])
def test_key_weights_problem_refused(lib, field, value):
    pr = grad_problem(**{field: value})
    n = ctypes.c_size_t(0)
    assert lib.slikl_key_weights_workspace_size(ctypes.byref(pr), ctypes.byref(n)) == INVALID
    assert weights_rc(lib, pr, weights_tensors()) == INVALID


def test_key_weights_refused(lib):
    pr = grad_problem(dtype=9, N1=0, D=5, deterministic=7)      # not read
    tn = weights_tensors()
    need = sli.slikl_key_weights_workspace_size(pr)
    assert passes(weights_rc, lib, pr, tn, n=need)
    assert weights_rc(lib, pr, tn, n=need - 1) == sli.SLIKL_ERR_WORKSPACE_TOO_SMALL
    assert weights_rc(lib, pr, tn, ws=None) == NULLPTR
    assert weights_rc(lib, pr, tn, ws=ctypes.c_void_p((1 << 30) + 8)) == INVALID
    for decay in (-0.5, float("nan"), float("inf")):
        assert weights_rc(lib, pr, tn, decay=decay) == INVALID
    for name in ("sparse_indices", "weights", "out"):
        t = weights_tensors()
        setattr(t, name, None)
        assert weights_rc(lib, pr, t) == NULLPTR, name
    for name in ("sparse_indices", "weights", "scores", "out", "status"):
        t = weights_tensors()
        setattr(t, name, 0x10002)
        assert weights_rc(lib, pr, t) == INVALID, name
    for side_ in ("q", "k"):
        p2 = grad_problem(**{"layout_" + side_: sli.SLIKL_TND, "T1": 32, "T2": 32})
        assert weights_rc(lib, p2, tn) == NULLPTR
    assert weights_rc(lib, pr, tn, opt=ctypes.byref(sli.make_options(seq_used_q=0x1002))) == INVALID
    assert lib.slikl_key_weights_workspace_size(ctypes.byref(pr), None) == sli.SLIKL_ERR_INNER_NULLPTR
    assert lib.slikl_key_weights(None, ctypes.byref(tn), 1.0, WS, 1 << 40, None, None) == NULLPTR


def evict_call():
    pr = sli.slikl_evict_problem(sli.SLIKL_BSND, 2, 2, 100, 0, 10, 2, 3)
    tn = sli.slikl_evict_tensors(0x10000, None, None, 0x20000, 0x30000, 0x40000, 0x50000)
    tn.caches[0] = (0x100000, 0x200000, 256)
    tn.caches[1] = (0x300000, 0x400000, 16)
    return pr, tn


def evict_rc(lib, pr, tn):
    return lib.slikl_evict(ctypes.byref(pr), ctypes.byref(tn), None)


@pytest.mark.parametrize("field,value", [
    ("layout_k", 2), ("n_caches", -1), ("n_caches", 9), ("B", 0), ("S2", 0), ("S2", 1 << 31), ("budget", 0),
    ("budget", 1 << 31), ("budget", 1 << 30), ("sinks", -1), ("recent", -1), ("sinks", 8), ("recent", 9),
    ("sinks", 1 << 62), ("B", 1 << 31),
])
def test_evict_problem_refused(lib, field, value):
    pr, tn = evict_call()
    assert passes(evict_rc, lib, pr, tn)
    setattr(pr, field, value)
    assert evict_rc(lib, pr, tn) == INVALID


def test_evict_tensors_refused(lib):
    for name in ("scores", "kept", "lengths"):
        pr, tn = evict_call()
        setattr(tn, name, None)
        assert evict_rc(lib, pr, tn) == NULLPTR, name
    for name in ("scores", "kept", "lengths", "scores_out", "status", "seq_used_k"):
        pr, tn = evict_call()
        setattr(tn, name, 0x10002)
        assert evict_rc(lib, pr, tn) == INVALID, name
    pr, tn = evict_call()
    pr.layout_k, pr.T2 = sli.SLIKL_TND, 200
    assert evict_rc(lib, pr, tn) == NULLPTR              # no cu_seqlens_k
    # out on in of the same or another cache, out on out, the scores on themselves
    for cache in ((0x100000, 0x100000, 256), (0x100000, 0x300000 + 200 * 16 - 16, 256), (0x100000, 0x400000, 256),
                  (0x100008, 0x200000, 256), (0x100000, 0x200008, 256), (0x100000, 0x200000, 24), (0x100000, 0x200000, 0),
                  (0x100000, 0x200000, -16)):
        pr, tn = evict_call()
        tn.caches[0] = cache
        assert evict_rc(lib, pr, tn) == INVALID, cache
    for cache in ((None, 0x200000, 256), (0x100000, None, 256)):
        pr, tn = evict_call()
        tn.caches[0] = cache
        assert evict_rc(lib, pr, tn) == NULLPTR, cache
    pr, tn = evict_call()
    tn.scores_out = 0x10000 + 4 * 199
    assert evict_rc(lib, pr, tn) == INVALID
    pr, tn = evict_call()
    tn.scores_out = None
    assert passes(evict_rc, lib, pr, tn)


def test_evict_refuses_outputs_over_other_tensors(lib):
    """The rows of `kept` are followed wherever they lead, and scores are read while rows are chosen: no
    output may share a byte with an input or with another output, whichever they are."""
    def call(tnd):
        pr, tn = evict_call()
        tn.seq_used_k = 0x60000
        if tnd:
            pr.layout_k, pr.S2, pr.T2, tn.cu_seqlens_k = sli.SLIKL_TND, 0, 200, 0x70000
        return pr, tn

    outs = {"kept": 80, "lengths": 8, "scores_out": 80, "status": 4, 0: 20 * 256, 1: 20 * 16}
    ins = {"scores": 800, "seq_used_k": 8, "cu_seqlens_k": 12, 0: 200 * 256, 1: 200 * 16}

    def at(tn, name, out):
        if isinstance(name, str):
            return getattr(tn, name)
        return tn.caches[name].out if out else tn.caches[name].in_

    def move(tn, name, to):
        if isinstance(name, str):
            setattr(tn, name, to)
        else:
            tn.caches[name].out = to

    for tnd in (False, True):
        assert passes(evict_rc, lib, *call(tnd))
        for o, size in outs.items():
            step = 4 if isinstance(o, str) else 16           # keeps it aligned
            others = [(n, s, True) for n, s in outs.items() if n != o] + [(n, s, False) for n, s in ins.items()]
            for name, n, is_out in others:
                if name == "cu_seqlens_k" and not tnd:
                    continue                                 # not there
                pr, tn = call(tnd)
                there = at(tn, name, is_out)
                last = (there + n - 1) // step * step        # shares the last bytes, shares the first ones
                first = there - (size - 1) // step * step
                for to in (there, last, first):
                    if (o, name, to) == ("lengths", "seq_used_k", there):
                        continue                             # allowed: in place
                    pr, tn = call(tnd)
                    move(tn, o, to)
                    assert evict_rc(lib, pr, tn) == INVALID, (o, name, hex(to))
        pr, tn = call(tnd)
        tn.lengths = tn.seq_used_k
        assert passes(evict_rc, lib, pr, tn)
        pr, tn = call(tnd)                                   # next to one another is not over one another
        tn.lengths, tn.scores_out = tn.kept + 80, tn.kept + 88
        assert passes(evict_rc, lib, pr, tn)


def test_binding_refuses_before_any_launch():
    """Wrong types, shapes and devices raise ValueError, on the CPU too."""
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sli.qk_norm_rope(x, None)                                   # not on a GPU
    with pytest.raises(ValueError):
        sli.qk_norm_rope(None, None)
    with pytest.raises(ValueError):
        sli.checkpoint_pack(x)
    with pytest.raises(ValueError):
        sli.checkpoint_unpack(sli.Checkpoint(x.to(torch.float8_e4m3fn), torch.zeros(1, 4, 2), torch.bfloat16))
    with pytest.raises(ValueError):
        sli.key_weights(torch.zeros(1, 1, 1, 4), torch.zeros(1, 1, 1, 4, dtype=torch.int32), torch.zeros(1, 4))
    with pytest.raises(ValueError):
        sli.evict(torch.zeros(1, 4), [], 2)
    for bad in (x.expand(3, 4, 2, 64)[:, :1], x.transpose(1, 2), x[..., ::2], torch.zeros(4, 2, 65)[..., :64],
                torch.zeros(4, 1, 64).expand(4, 2, 64), torch.zeros(1, 2, 64).expand(4, 2, 64),
                torch.zeros(2, 5, 2, 64)[:, :4], torch.zeros(4, 132).view(4, 132)[:, :128].unflatten(1, (2, 64))):
        with pytest.raises(ValueError):
            sli._load_binding().row_stride(bad, "x")
    ok = torch.zeros(4, 200)[:, 8:136].unflatten(1, (2, 64))
    assert sli._load_binding().row_stride(ok, "x") == 200 and sli._load_binding().row_stride(x, "x") == 128
    assert sli._load_binding().row_stride(torch.zeros(1, 1, 2, 64).expand(1, 1, 2, 64), "x") == 128


def test_the_library_builds_without_torch(lib, tmp_path):
    """A C user needs no torch: without it the build makes the library, says so, and succeeds."""
    code = ("import importlib.util, sys\n"
            f"spec = importlib.util.spec_from_file_location('b', {slibuild.__file__!r})\n"
            "b = importlib.util.module_from_spec(spec)\n"
            "spec.loader.exec_module(b)\n"
            f"b.TORCH_LIB = {str(tmp_path / '_slikl_torch.so')!r}\n"
            "assert importlib.util.find_spec('torch') is None\n"
            "print(b.build())\n")
    r = subprocess.run([sys.executable, "-I", "-S", "-c", code], capture_output=True, text=True, cwd=tmp_path)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == slibuild.LIB and "torch" in r.stderr and not os.listdir(tmp_path)


def test_the_binding_is_built_anew_for_another_torch(lib, tmp_path, monkeypatch):
    """File times do not tell that torch or Python changed; what the module was built for does."""
    built = []

    def run(cmd, **kw):
        built.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(slibuild, "TORCH_LIB", str(tmp_path / "_slikl_torch.so"))
    monkeypatch.setattr(slibuild, "OBJDIR", str(tmp_path))
    monkeypatch.setattr(slibuild.subprocess, "run", run)
    version = importlib.metadata.version
    for torch_version, count in (("2.11.0", 1), ("2.11.0", 1), ("2.12.0", 2), ("2.12.0", 2), ("2.11.0", 3)):
        monkeypatch.setattr(importlib.metadata, "version",
                            lambda name, v=torch_version: v if name == "torch" else version(name))
        assert slibuild.build_torch() == slibuild.TORCH_LIB
        assert len(built) == count, torch_version
    slibuild.build_torch(force=True)
    assert len(built) == 4

    def unknown(name):
        raise importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(importlib.metadata, "version", unknown)
    slibuild.build_torch()
    slibuild.build_torch()
    assert len(built) == 5


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_layouts_match_a_c_caller(lib, tmp_path):
    libdir = os.path.dirname(lib._name)
    exe = str(tmp_path / "c_caller_operators")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c_caller_operators.c"), "-o", exe, "-L", libdir, "-lslikl",
                    "-Wl,-rpath," + libdir], check=True, capture_output=True, text=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines()
    sizes, rcs = 0, []
    for line in lines:
        parts = line.split()
        if parts[0] == "size":
            assert ctypes.sizeof(getattr(sli, parts[1])) == int(parts[2]), parts[1]
            sizes += 1
        elif parts[0] == "field":
            name = "in_" if parts[2] == "in" else parts[2]
            assert getattr(getattr(sli, parts[1]), name).offset == int(parts[3]), line
        else:
            rcs.append((int(parts[1]), int(parts[2])))
    assert sizes == 8
    qk = sli.slikl_qk_problem(sli.SLIKL_BF16, 0, 128, 64, 4096, 1e-6, 0, side(4096, 4096, 64),
                              side(4096, 4096, 1, norm=sli.SLIKL_NORM_LAYER))
    pr = sli.slikl_problem(sli.SLIKL_BF16, 0, 0, 0, 1, 4096, 4096, 0, 0, 64, 128, 2048)
    assert rcs == [(0, sli.slikl_qk_norm_rope_grad_workspace_size(qk)),
                   (0, sli.slikl_grad_projected_workspace_size(pr, qk)), (0, sli.slikl_key_weights_workspace_size(pr))]
