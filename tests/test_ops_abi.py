"""Struct layouts and host-side refusals of the calls around the layer (CPU: nothing is launched)."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

import tile_sparse_video_pack_b200 as T
from tile_sparse_video_pack_b200 import vsa as V

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"vsa_strides": V.VsaStrides, "vsa_norm_rope": V.VsaNormRope, "vsa_linear_args": V.VsaLinearArgs,
           "vsa_linear_grad_args": V.VsaLinearGradArgs}


def test_struct_layouts_match_c():
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "vsa.h"\nint main(void) {' + "\n".join(lines) + "return 0;}"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "p.c"), os.path.join(d, "p")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for cls in STRUCTS.values():
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def test_enumerations_match_header():
    text = open(os.path.join(ROOT, "include", "vsa.h")).read()
    for name, value in (("VSA_ROPE_INTERLEAVED", V.ROPE_LAYOUTS["interleaved"]), ("VSA_ROPE_HALVES", V.ROPE_LAYOUTS["halves"]),
                        ("VSA_ACT_NONE", V.ACTIVATIONS["none"]), ("VSA_ACT_GELU_TANH", V.ACTIVATIONS["gelu_tanh"]),
                        ("VSA_ACT_SILU", V.ACTIVATIONS["silu"])):
        assert f"{name} = {value}" in text


def test_norm_rope_refusals():
    w, t = torch.ones(64), torch.ones(8, 32)
    with pytest.raises(ValueError):
        T.NormRope(w, w, layout="pairs")
    with pytest.raises(ValueError):
        T.NormRope(w, w, cos=t)
    with pytest.raises(ValueError):
        T.NormRope(w, torch.ones(2, 64))
    assert T.NormRope(torch.ones(2, 64), None).per_head and not T.NormRope(w, None).per_head
    assert not T.NormRope(cos=t, sin=t).per_head


def test_calls_refuse_cpu_tensors_before_any_launch():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    V.library()
    with pytest.raises(TypeError):
        V._matrix(x, 64, "x", 0)
    with pytest.raises(TypeError):
        V._addr(x, torch.bfloat16, "x", 0)
    with pytest.raises(TypeError):
        V._addr([1, 2], torch.bfloat16, "x", 0)
    assert V._addr(None, torch.bfloat16, "x", 0) is None


def test_activation_and_gate_shapes():
    with pytest.raises(ValueError):
        T.Plan._act("tanh")
    for shape in ((3, 64), (2, 32), (64,), (0, 64)):
        with pytest.raises(ValueError):
            T.Plan._gate(torch.zeros(shape), 8, 64, 0)
    assert T.Plan._gate(None, 8, 64, 0) == (None, 0)


def test_an_output_beside_the_input_is_taken_and_one_over_it_refused():
    from tile_sparse_video_pack_b200.layer import _keeps
    wide = torch.zeros(2, 6, 96, dtype=torch.bfloat16)
    x = wide[..., 16:48]
    for out in (wide[..., 48:], wide[..., :16], wide[..., 72:80], torch.zeros(2, 6, 32, dtype=torch.bfloat16), None, wide[:0]):
        _keeps(x, out, True)
    _keeps(wide[:1, :, :32], wide[1:, :, :32], True)
    for out in (x, wide[..., :24], wide[..., 40:72], wide[..., 47:48], wide[:1, 3:4, 16:24], wide.view(-1)[16:24],
                wide[..., 0:96], wide.view(2, 12, 48)[:, ::2]):
        _keeps(x, out, False)
        with pytest.raises(ValueError):
            _keeps(x, out, True)
    with pytest.raises(ValueError):      # rows that wrap into the next one's columns
        _keeps(wide.view(-1)[80:176].view(1, 96), wide.view(-1)[96:128].view(1, 32), True)


def test_blocks_refuse_biases_of_another_length():
    """The direct path slices b_qkv: a longer one would have been taken without a word."""
    from types import SimpleNamespace as NS
    layer = NS(plan=NS(desc=NS(heads=2, head_dim=64)))
    w_qkv, w_out, norm = torch.zeros(384, 96), torch.zeros(80, 128), T.NormRope()
    T.TileSparseBlock(layer, w_qkv, w_out, norm, torch.zeros(384), torch.zeros(80))
    T.FeedForward(None, w_qkv, torch.zeros(96, 384), torch.zeros(384), torch.zeros(96))
    for b in (torch.zeros(392), torch.zeros(376), torch.zeros(1, 384)):
        with pytest.raises(ValueError):
            T.TileSparseBlock(layer, w_qkv, w_out, norm, b)
        with pytest.raises(ValueError):
            T.FeedForward(None, w_qkv, torch.zeros(96, 384), b)
    for b in (torch.zeros(128), torch.zeros(80, 1)):
        with pytest.raises(ValueError):
            T.TileSparseBlock(layer, w_qkv, w_out, norm, None, b)
        with pytest.raises(ValueError):
            T.FeedForward(None, w_qkv, torch.zeros(96, 384), None, b)
