"""Refusals, limits and size helpers of the products, block norms and clipping, and
what their machine code relies on, without a GPU.

No call here enqueues device work: each is pure host code or must be rejected by
validation before any HIP call."""
import ctypes
import math
import os
import re
import subprocess

import pytest

from mixture_experts_layer_up_amd import binding, build
from mixture_experts_layer_up_amd.binding import Gradient, LinearShape, NormGradients, NormShape

OK, INVALID, SHAPE, WS, ALIGN = 0, -1, -2, -3, -4
ref = ctypes.byref
BIG = 1 << 40
P = 1 << 20      # an aligned address; never dereferenced: validation rejects first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        build.build(verbose=False)
    return binding.load_library()


@pytest.mark.parametrize("cname,cls", [
    ("moe_lora_linear_shape", "LinearShape"), ("moe_lora_norm_shape", "NormShape"),
    ("moe_lora_norm_gradients", "NormGradients"), ("moe_lora_gradient", "Gradient")])
def test_ctypes_structs_match_header(cname, cls):
    text = re.sub(r"/\*.*?\*/", "", open(binding.HEADER_PATH).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (cname, cname), text, re.S).group(1)
    kinds = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float}
    fields = []
    for d in (d.strip() for d in body.split(";") if d.strip()):
        name = re.search(r"(\w+)$", d).group(1)
        fields.append((name, ctypes.c_void_p if "*" in d else kinds[d.split()[0]]))
    assert fields == list(getattr(binding, cls)._fields_)


def test_names_match_header():
    text = open(binding.HEADER_PATH).read()
    for prefix, names in (("ACT", binding.ACTIVATIONS), ("GATE", binding.GATES)):
        defs = {n.lower(): int(v) for n, v in re.findall(r"#define MOE_LORA_%s_(\w+)\s+(\d+)" % prefix, text)}
        assert defs == {n: i for i, n in enumerate(names)}


# ---------------------------------------------------------------- products

BAD_LINEAR = [(dict(rows=-1), SHAPE), (dict(rows=(1 << 24) + 1), SHAPE), (dict(in_features=0), SHAPE),
              (dict(in_features=12), SHAPE), (dict(in_features=131080), SHAPE), (dict(out_features=0), SHAPE),
              (dict(out_features=131073), SHAPE), (dict(rows=1 << 24, out_features=8192), SHAPE),
              (dict(activation=5), INVALID), (dict(activation=-1), INVALID), (dict(out_fp32=2), INVALID)]


def _linear_shape(**over):
    base = dict(rows=100, in_features=64, out_features=48, activation=0, out_fp32=0)
    base.update(over)
    return LinearShape(*[base[n] for n, _ in LinearShape._fields_])


def _linear(lib, s, x=P, w=P, bias=None, residual=None, out=P, preact=None, ws=P, n=BIG):
    return lib.moe_lora_linear(ref(s) if s is not None else None, x, w, bias, residual, out, preact, ws, n, None)


def _linear_grad(lib, s, x=P, w=P, preact=P, d_out=P, d_x=P, d_w=P, d_bias=P, ws=P, n=BIG):
    return lib.moe_lora_linear_backward(ref(s) if s is not None else None, x, w, preact, d_out, d_x, d_w, d_bias,
                                        ws, n, None)


@pytest.mark.parametrize("over,rc", BAD_LINEAR)
def test_bad_linear_shapes(lib, over, rc):
    s = _linear_shape(**over)
    assert _linear(lib, s) == rc and _linear_grad(lib, s) == rc
    assert binding.linear_workspace_size(s) == 0 and binding.linear_backward_workspace_size(s) == 0


def test_linear_arguments(lib):
    s = _linear_shape(rows=60000, out_features=49)    # needs a workspace: a padded weight
    assert _linear(lib, None) == INVALID and _linear_grad(lib, None) == INVALID
    for name in ("x", "w", "out", "ws"):
        assert _linear(lib, s, **{name: None}) == INVALID
    for name, off in (("x", 2), ("w", 8), ("bias", 2), ("residual", 1), ("out", 1), ("preact", 1), ("ws", 16)):
        assert _linear(lib, s, **{name: P + off}) == ALIGN
    assert _linear(lib, _linear_shape(out_fp32=1), out=P + 2) == ALIGN
    need = binding.linear_workspace_size(s)
    assert need >= 64 * 56 * 2 and _linear(lib, s, n=need - 1) == WS
    assert _linear(lib, _linear_shape(rows=0), x=None, w=None, out=None, ws=None, n=0) == OK


def test_linear_backward_arguments(lib):
    s = _linear_shape(activation=3)
    assert _linear_grad(lib, s, d_x=None, d_w=None, d_bias=None) == INVALID
    for name in ("preact", "d_out", "ws"):
        assert _linear_grad(lib, s, **{name: None}) == INVALID
    assert _linear_grad(lib, s, w=None) == INVALID and _linear_grad(lib, s, x=None) == INVALID
    assert _linear_grad(lib, s, w=None, d_x=None, n=0) == WS        # w is then not needed
    assert _linear_grad(lib, s, x=None, d_w=None, n=0) == WS
    for name, off in (("x", 8), ("w", 8), ("d_out", 8), ("d_x", 8), ("d_w", 8), ("preact", 1), ("d_bias", 2),
                      ("ws", 128)):
        assert _linear_grad(lib, s, **{name: P + off}) == ALIGN
    need = binding.linear_backward_workspace_size(s)
    assert _linear_grad(lib, s, n=need - 1) == WS
    # no rows: the inputs may be missing, the weight's gradient is still written
    assert _linear_grad(lib, _linear_shape(rows=0), x=None, w=None, preact=None, d_out=None, n=0) == WS


def test_linear_workspaces_grow(lib):
    """Split sums are bounded; dz and a padded weight are there when they are needed."""
    for N in (48, 49, 2048):
        for act in range(5):
            for rows in (0, 1, 64, 65, 4096, 65536):
                s = _linear_shape(rows=rows, in_features=2048, out_features=N, activation=act)
                W = -(-N // 8) * 8 * (2 if act == 4 else 1)
                fwd, bwd = binding.linear_workspace_size(s), binding.linear_backward_workspace_size(s)
                assert fwd % 256 == 0 and bwd % 256 == 0 and fwd <= 2048 * W * 2 + (600 << 20)
                if act or N == 49:
                    assert bwd >= rows * W * 2
                if rows <= 64:      # one launch, w as it is
                    assert fwd == 0


# ---------------------------------------------------------------- norms

BAD_NORM = [(dict(rows=-1), SHAPE), (dict(rows=(1 << 24) + 1), SHAPE), (dict(hidden=0), SHAPE),
            (dict(hidden=96), SHAPE), (dict(hidden=65600), SHAPE), (dict(eps=0.0), INVALID),
            (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
            (dict(residual_scale=math.inf), INVALID), (dict(weight_offset=math.nan), INVALID),
            (dict(gate=3), INVALID), (dict(gate=-1), INVALID)]


def _norm_shape(**over):
    base = dict(rows=10, hidden=128, eps=1e-6, residual_scale=1.0, weight_offset=0.0, gate=0)
    base.update(over)
    return NormShape(*[base[n] for n, _ in NormShape._fields_])


def _norm(lib, s, x=P, y=P, w_post=P, w_pre=P, gate=None, r=P, z=P):
    return lib.moe_lora_block_norm(ref(s) if s is not None else None, x, y, w_post, w_pre, gate, r, z, None)


def _norm_grad(lib, s, r=P, y=P, w_post=P, w_pre=P, gate=None, d_r=P, d_z=P, ws=P, n=BIG, none=False, **over):
    d = dict(d_residual=P, d_branch=P, d_post_weight=P, d_pre_weight=P, d_gate=P if gate else None)
    d.update(over)
    g = None if none else ref(NormGradients(*[d[k] for k, _ in NormGradients._fields_]))
    return lib.moe_lora_block_norm_backward(ref(s) if s is not None else None, r, y, w_post, w_pre, gate, d_r, d_z,
                                            g, ws, n, None)


@pytest.mark.parametrize("over,rc", BAD_NORM)
def test_bad_norm_shapes(lib, over, rc):
    s = _norm_shape(**over)
    assert _norm(lib, s) == rc and _norm_grad(lib, s) == rc
    assert binding.block_norm_backward_workspace_size(s) == 0


def test_norm_arguments(lib):
    s = _norm_shape()
    assert _norm(lib, None) == INVALID
    for over in (dict(x=None, y=None), dict(r=None, z=None), dict(z=None), dict(w_pre=None), dict(gate=P),
                 dict(y=None), dict(x=None, y=None, w_post=None)):
        assert _norm(lib, s, **over) == INVALID
    for name in ("x", "y", "w_post", "w_pre", "r", "z"):
        assert _norm(lib, s, **{name: P + 8}) == ALIGN
    token, channel = _norm_shape(gate=1), _norm_shape(gate=2)
    assert _norm(lib, token) == INVALID and _norm(lib, channel) == INVALID
    assert _norm(lib, token, gate=P + 2) == ALIGN and _norm(lib, channel, gate=P + 8) == ALIGN
    assert _norm(lib, channel, y=None, w_post=None, gate=P) == INVALID
    assert _norm(lib, _norm_shape(rows=0), x=None, y=None, r=None, z=None) == OK


def test_norm_backward_arguments(lib):
    s = _norm_shape()
    assert _norm_grad(lib, None) == INVALID and _norm_grad(lib, s, none=True) == INVALID
    none = dict(d_residual=None, d_branch=None, d_post_weight=None, d_pre_weight=None)
    for over in (none, dict(d_r=None, d_z=None), dict(gate=P), dict(w_pre=None), dict(r=None), dict(d_z=None),
                 dict(w_post=None), dict(y=None), dict(ws=None), dict(d_gate=P)):
        assert _norm_grad(lib, s, **over) == INVALID
    for name in ("r", "y", "w_post", "w_pre", "d_r", "d_z", "d_residual", "d_branch"):
        assert _norm_grad(lib, s, **{name: P + 8}) == ALIGN
    for name in ("d_post_weight", "d_pre_weight"):
        assert _norm_grad(lib, s, **{name: P + 2}) == ALIGN
    assert _norm_grad(lib, s, ws=P + 64) == ALIGN
    assert _norm_grad(lib, s, n=binding.block_norm_backward_workspace_size(s) - 1) == WS
    # without d_normed its weight and new_residual are not needed
    assert _norm_grad(lib, s, d_z=None, w_pre=None, r=None, d_pre_weight=None, n=0) == WS
    assert _norm_grad(lib, _norm_shape(gate=1), gate=P, w_post=None, d_post_weight=None, y=None) == INVALID


def test_norm_workspace_is_bounded(lib):
    """Column sums of as many blocks as run at once; of wide rows 16 bytes each too."""
    for H, most in ((64, 512), (2048, 512), (4160, 256), (8192, 256), (8256, 128), (65536, 128)):
        rows = (0, 1, 100, 10000, 1 << 24)
        sizes = [binding.block_norm_backward_workspace_size(_norm_shape(rows=T, hidden=H)) for T in rows]
        assert sizes == sorted(sizes) and sizes[0] >= 3 * H * 4
        for T, size in zip(rows, sizes):
            assert size <= most * 3 * H * 4 + (16 * T + 256 if H > 8192 else 0)


# ---------------------------------------------------------------- clipping

def _clip(lib, entries, max_norm=1.0, norm=P, ws=P, n=BIG, count=None):
    table = (Gradient * max(1, len(entries)))(*[Gradient(*e) for e in entries])
    return lib.moe_lora_clip_gradients(table, len(entries) if count is None else count, max_norm, norm, ws, n, None)


def test_clip_arguments(lib):
    a, b = 1 << 21, 1 << 22
    ok = [(a, a, 100, 0, 0), (b, b, 100, 1, 0)]
    for entries, rc in ((ok, WS), ([(a, a, -1, 0, 0)], SHAPE), ([(a, a, 1 << 36, 0, 0)], SHAPE),
                        ([(a, a, 10, 2, 0)], INVALID), ([(a, a, 10, 0, 1)], INVALID), ([(None, a, 10, 0, 0)], INVALID),
                        ([(a, None, 10, 0, 0)], INVALID), ([(a + 1, a + 1, 10, 0, 0)], ALIGN),
                        ([(a + 2, a + 2, 10, 1, 0)], ALIGN), ([(a, a + 2000 + 2, 10, 1, 0)], ALIGN),
                        ([(None, None, 0, 0, 0)], WS)):
        assert _clip(lib, entries, n=0) == rc
    assert _clip(lib, ok, norm=None) == INVALID and _clip(lib, ok, norm=P + 2) == ALIGN
    assert _clip(lib, ok, ws=None) == INVALID and _clip(lib, ok, ws=P + 8) == ALIGN
    for bad in (-1.0, -math.inf, math.nan):
        assert _clip(lib, ok, bad) == INVALID
    assert _clip(lib, [(a, None, 10, 0, 0)], math.inf, n=0) == WS       # the norm only needs no out
    assert _clip(lib, ok, count=-1) == SHAPE and _clip(lib, ok, count=4097) == SHAPE
    assert lib.moe_lora_clip_gradients(None, 2, 1.0, P, P, BIG, None) == INVALID


def test_clip_overlaps(lib):
    """Ranges of two tensors that meet, in any order; neighbours do not."""
    a = 1 << 21
    meet = [[(a, a, 100, 0, 0), (a, a, 100, 0, 0)], [(a, a, 100, 0, 0), (a + 198, a + 198, 1, 0, 0)],
            [(a + 198, a + 198, 5, 0, 0), (a, a, 100, 0, 0)], [(a, 2 * a, 100, 0, 0), (3 * a, a, 100, 0, 0)],
            [(a, a + 100, 100, 0, 0)], [(a, a, 100, 1, 0), (a + 396, a + 396, 100, 0, 0)]]
    apart = [[(a, a, 100, 0, 0), (a + 200, a + 200, 100, 0, 0)], [(a + 200, a + 200, 9, 0, 0), (a, a, 100, 0, 0)],
             [(a, 2 * a, 100, 0, 0), (3 * a, 4 * a, 100, 0, 0)], [(a, a, 0, 0, 0), (a, a, 100, 0, 0)]]
    for entries in meet:
        assert _clip(lib, entries, n=0) == INVALID
    for entries in apart:
        assert _clip(lib, entries, n=0) == WS
    every = [(a + 1000 * i, a + 1000 * i, 250, 1, 0) for i in range(4096)]
    assert _clip(lib, every, n=0) == WS and _clip(lib, every[::-1], n=0) == WS
    every[4000] = every[17]
    assert _clip(lib, every, n=0) == INVALID


def test_clip_workspace(lib):
    """A sum for each block: of 2048 to 32768 elements, by how many there are in all."""
    for sizes, chunk in (([0], 2048), ([1], 2048), ([2048], 2048), ([2049, 7], 2048), ([1 << 21, 1], 4096),
                         ([1 << 26], 32768), ([5, 70000, 1 << 35], 32768)):
        table = (Gradient * len(sizes))(*[Gradient(4096, 4096, n, 0, 0) for n in sizes])
        chunks = sum(-(-n // chunk) for n in sizes)
        need = lib.moe_lora_clip_workspace_size(table, len(sizes))
        assert need == 256 + -(-chunks * 8 // 256) * 256


# ---------------------------------------------------------------- machine code

def _asm(name, tmp_path):
    src = os.path.join(build.CSRC, name)
    out = tmp_path / (name + ".s")
    subprocess.run([build.HIPCC, *build.COMMON_FLAGS, "--cuda-device-only", "-S", src, "-o", str(out)], check=True,
                   capture_output=True)
    return out.read_text()


def test_direct_loads_own_m0(tmp_path):
    """The direct loads set M0, which the compiler is not told about: nothing else uses it."""
    asm = _asm("linear_tile.hip", tmp_path)
    lines = [ln.split(";")[0].strip() for ln in asm.splitlines()]
    lines = [ln for ln in lines if ln and not ln.startswith(("#", "."))]
    loads = 0
    for a, b in zip(lines, lines[1:]):
        if re.search(r"\bm0\b", a):
            assert re.match(r"s_mov_b32 m0, ", a) and re.match(r"buffer_load_dwordx4 v\d+, s\[.*offen lds$", b), (a, b)
            loads += 1
        assert not re.match(r"(s_movrel|v_movrel|s_sendmsg|ds_gws|lds_param|v_interp)", a), a
    assert loads > 0


def test_matrix_instructions_see_every_lane(tmp_path):
    """MFMA ignores EXEC: none may sit where a branch has narrowed it."""
    from tests.test_isa_mfma_scalar_guards import _mfma_under_exec_mask
    for name in ("linear_tile.hip", "linear_rows.hip"):
        # the mask check reads a kernel to its first end: earlier ones become jumps out of it
        parts = re.split(r"(?m)^(\.Lfunc_end\d+:)", _asm(name, tmp_path))
        parts = [re.sub(r"s_endpgm(?=[\s\S]*s_endpgm)", "s_branch .LBB_out", part) for part in parts]
        bad, total = _mfma_under_exec_mask("".join(parts))
        assert total > 0 and not bad, bad[:5]


def test_sources_do_not_spill(tmp_path):
    """No scratch memory in the products' kernels."""
    for name in ("linear_tile.hip", "linear_rows.hip"):
        spills = re.findall(r"\.vgpr_spill_count:\s+(\d+)", _asm(name, tmp_path))
        assert spills and not any(int(s) for s in spills)
