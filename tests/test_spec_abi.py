"""libgdn_spec.so on the CPU: its symbols, its struct, and the host checks of
every entry point.  No kernel is launched: the calls below fail a check, or
pass them all on host tensors, which the binding then refuses."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import spec_plain
from gated_deltanet_recurrent_sigmoid_b200 import binding, build, speculative as spec

HEADER = os.path.join(build.INCLUDE, "gdn_spec.h")
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib(gdn_lib):
    return spec.load()


def test_exports_and_constants():
    text = open(HEADER).read()
    declared = set(re.findall(r"GDN_API\s+[\w\s\*]+?\b(gdn_\w+)\s*\(", text))
    assert declared == {"gdn_token_probs", "gdn_verify_drafts", "gdn_commit_states", "gdn_step_maps",
                        "gdn_spec_version"}
    nm = subprocess.run(["nm", "-D", "--defined-only", build.SPEC_LIB_PATH], capture_output=True, text=True,
                        check=True).stdout
    assert {l.split()[-1] for l in nm.splitlines() if " T " in l and "gdn" in l} == declared
    assert spec.load().gdn_spec_version() == int(re.search(r"GDN_SPEC_ABI_VERSION (\d+)", text).group(1))
    for name in ("BAD_SEQ", "BAD_TEMPERATURE", "BAD_TOKEN", "BAD_PROBS", "BAD_COUNT", "BAD_LENGTH", "BAD_BLOCKS",
                 "NO_ROOM"):
        bit = 1 << int(re.search(rf"#define GDN_DEV_{name}\s+\(1u << (\d+)\)", text).group(1))
        assert bit == getattr(spec, f"DEV_{name}") == getattr(spec_plain, f"DEV_{name}")
    assert spec.CHECK_ONLY == 1 << int(re.search(r"GDN_SPEC_CHECK_ONLY \(1u << (\d+)\)", text).group(1))
    assert spec.MAX_VOCAB == int(re.search(r"GDN_SPEC_MAX_VOCAB (\d+)", text).group(1))


def test_struct_layout_matches_a_c_compile(tmp_path):
    fields = [f[0] for f in spec.GdnStepMapsCall._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gdn_spec.h"\nint main(void) {\n' + "".join(
        f'printf("%zu ", offsetof(gdn_step_maps_call, {f}));\n' for f in fields) +
        'printf("%zu", sizeof(gdn_step_maps_call)); return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", build.INCLUDE, "-o", str(exe), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(spec.GdnStepMapsCall, f).offset for f in fields] + [ctypes.sizeof(spec.GdnStepMapsCall)]


def refused(code, make, **changes):
    """The call with ``changes`` fails with ``code``; without them it passes
    every check of the library and is refused for its host tensors only."""
    fn, args = make()
    with pytest.raises(ValueError):
        fn(**args)
    args.update(changes)
    with pytest.raises(binding.GdnError) as e:
        fn(**args)
    assert e.value.status == code, binding.status_string(e.value.status)


def make_probs(R=4, V=40, S=3):
    return spec.token_probs, dict(logits=torch.zeros(R, V), probs=torch.zeros(R, V), temperature=torch.ones(S),
                                  row_seq=torch.zeros(R, dtype=I32))


@pytest.mark.parametrize("code,changes", [
    (binding.ERR_DTYPE, dict(logits=torch.zeros(4, 40, dtype=torch.float16))),
    (binding.ERR_DTYPE, dict(probs=torch.zeros(4, 40, dtype=torch.float64))),
    (binding.ERR_DTYPE, dict(temperature=torch.ones(3, dtype=torch.float64))),
    (binding.ERR_DTYPE, dict(row_seq=torch.zeros(4, dtype=torch.int64))),
    (binding.ERR_SHAPE, dict(probs=torch.zeros(4, 41))),
    (binding.ERR_SHAPE, dict(logits=torch.zeros(40, 4).t())),
    (binding.ERR_SHAPE, dict(probs=torch.zeros(1, 40).expand(4, 40))),
    (binding.ERR_SHAPE, dict(row_seq=torch.zeros(5, dtype=I32))),
    (binding.ERR_SHAPE, dict(row_seq=torch.zeros(8, dtype=I32)[::2])),
    (binding.ERR_SHAPE, dict(row_seq=None)),                            # then one temperature a row
    (binding.ERR_NULL_ARG, dict(temperature=None)),                     # row_seq without temperatures
    (binding.ERR_SHAPE, dict(logits=torch.zeros(4, 0), probs=torch.zeros(4, 0))),
    (binding.ERR_UNSUPPORTED, dict(logits=torch.zeros(4, spec.MAX_VOCAB + 1), probs=torch.zeros(4, spec.MAX_VOCAB + 1))),
    (binding.ERR_ARG, dict(flags=1)),
])
def test_probs_refusals(code, changes):
    refused(code, make_probs, **changes)


def test_probs_refuses_overlap():
    both = torch.zeros(4, 40)
    refused(binding.ERR_ALIAS, make_probs, logits=both, probs=both)
    refused(binding.ERR_ALIAS, make_probs, logits=torch.zeros(4, 80)[:, :40], probs=both, temperature=both[0, :3])


def make_verify(N=3, D=2, V=40):
    return spec.verify_drafts, dict(
        target_probs=torch.zeros(N * (D + 1), V), draft_tokens=torch.zeros(N, D, dtype=I32),
        draft_probs=torch.zeros(N, D, V), uniforms=torch.zeros(N, D + 1), out_tokens=torch.zeros(N, D + 1, dtype=I32),
        num_tokens=torch.zeros(N, dtype=I32), cu_seqlens=torch.zeros(N + 1, dtype=I32))


@pytest.mark.parametrize("code,changes", [
    (binding.ERR_DTYPE, dict(target_probs=torch.zeros(9, 40, dtype=torch.float16))),
    (binding.ERR_DTYPE, dict(draft_probs=torch.zeros(3, 2, 40, dtype=torch.bfloat16))),
    (binding.ERR_DTYPE, dict(draft_tokens=torch.zeros(3, 2, dtype=torch.int64))),
    (binding.ERR_DTYPE, dict(uniforms=torch.zeros(3, 3, dtype=torch.float64))),
    (binding.ERR_SHAPE, dict(uniforms=torch.zeros(3, 2))),
    (binding.ERR_SHAPE, dict(out_tokens=torch.zeros(3, 2, dtype=I32))),
    (binding.ERR_SHAPE, dict(num_tokens=torch.zeros(2, dtype=I32))),
    (binding.ERR_SHAPE, dict(draft_probs=torch.zeros(3, 3, 40))),
    (binding.ERR_SHAPE, dict(draft_probs=torch.zeros(3, 2, 41))),
    (binding.ERR_SHAPE, dict(cu_seqlens=torch.zeros(3, dtype=I32))),
    (binding.ERR_SHAPE, dict(cu_seqlens=None)),                         # then [N, T, vocab]
    (binding.ERR_SHAPE, dict(cu_seqlens=None, target_probs=torch.zeros(3, 4, 40))),     # T > D + 1
    (binding.ERR_SHAPE, dict(target_probs=torch.zeros(40, 9).t())),
    (binding.ERR_SHAPE, dict(state_indices=torch.zeros(4, dtype=I32))),
    (binding.ERR_SHAPE, dict(out_tokens=torch.zeros(1, 3, dtype=I32).expand(3, 3))),
    (binding.ERR_SHAPE, dict(num_tokens=torch.zeros(1, dtype=I32).expand(3))),
    (binding.ERR_ARG, dict(flags=binding.WRITE_INTERMEDIATE)),
])
def test_verify_refusals(code, changes):
    refused(code, make_verify, **changes)


def test_verify_refuses_overlap():
    both = torch.zeros(3, 3, dtype=I32)
    refused(binding.ERR_ALIAS, make_verify, out_tokens=both, draft_tokens=both[:, :2])
    refused(binding.ERR_ALIAS, make_verify, out_tokens=both, num_tokens=both[:, 0])


def make_commit(N=3, T=2, HV=2, slots=5):
    return spec.commit_states, dict(
        intermediate_states=torch.zeros(N * T, HV, 128, 128), num_tokens=torch.zeros(N, dtype=I32),
        state_pool=torch.zeros(slots, HV, 128, 128), state_indices=torch.arange(N, dtype=I32))


@pytest.mark.parametrize("code,changes", [
    (binding.ERR_DTYPE, dict(state_pool=torch.zeros(5, 2, 128, 128, dtype=torch.bfloat16))),
    (binding.ERR_SHAPE, dict(state_pool=torch.zeros(5, 3, 128, 128))),
    (binding.ERR_SHAPE, dict(intermediate_states=torch.zeros(7, 2, 128, 128))),          # not N * T rows
    (binding.ERR_SHAPE, dict(num_tokens=torch.zeros(2, dtype=I32))),
    (binding.ERR_SHAPE, dict(state_pool=torch.zeros(5, 2, 128, 128).transpose(2, 3))),
    (binding.ERR_SHAPE, dict(state_pool=torch.zeros(1, 2, 128, 128).expand(5, 2, 128, 128))),
    (binding.ERR_UNSUPPORTED, dict(state_pool=torch.zeros(5, 2, 64, 64), intermediate_states=torch.zeros(6, 2, 64, 64))),
    (binding.ERR_ALIGN, dict(state_pool=torch.zeros(5 * 2 * 128 * 128 + 1)[1:].view(5, 2, 128, 128))),
    (binding.ERR_SHAPE, dict(cu_seqlens=torch.zeros(3, dtype=I32))),
    (binding.ERR_ARG, dict(flags=binding.CHECK_INDICES)),
])
def test_commit_refusals(code, changes):
    refused(code, make_commit, **changes)


def test_commit_refuses_overlap():
    both = torch.zeros(8, 2, 128, 128)
    refused(binding.ERR_ALIAS, make_commit, intermediate_states=both[:6], state_pool=both[3:])


def make_maps(N=3, C=20, B=4, F=9):
    z = lambda *s: torch.zeros(*s, dtype=I32)  # noqa: E731
    return spec.step_maps, dict(
        lengths=z(N), context=z(N), slots=z(N), cu_seqlens=z(N + 1), state_indices=z(N), row_seq=z(C), positions=z(C),
        block_tables=z(N, B), blocks_held=z(N), free_blocks=z(F), free_head=z(1), blocks_held_out=z(N),
        free_head_out=z(1), slot_map=torch.zeros(C, dtype=torch.int64), block_size=16)


@pytest.mark.parametrize("code,changes", [
    (binding.ERR_DTYPE, dict(lengths=torch.zeros(3, dtype=torch.int64))),
    (binding.ERR_DTYPE, dict(slot_map=torch.zeros(20, dtype=I32))),
    (binding.ERR_SHAPE, dict(context=torch.zeros(4, dtype=I32))),
    (binding.ERR_SHAPE, dict(cu_seqlens=torch.zeros(3, dtype=I32))),
    (binding.ERR_SHAPE, dict(positions=torch.zeros(21, dtype=I32))),
    (binding.ERR_SHAPE, dict(block_tables=torch.zeros(4, 4, dtype=I32))),
    (binding.ERR_SHAPE, dict(block_tables=torch.zeros(4, 3, dtype=I32).t())),
    (binding.ERR_SHAPE, dict(block_tables=torch.zeros(1, 4, dtype=I32).expand(3, 4))),
    (binding.ERR_SHAPE, dict(free_head=torch.zeros(2, dtype=I32))),
    (binding.ERR_NULL_ARG, dict(slot_map=None)),
    (binding.ERR_NULL_ARG, dict(slots=None)),
    (binding.ERR_ARG, dict(block_size=0)),
    (binding.ERR_ARG, dict(flags=binding.NO_FINAL_WRITEBACK)),
])
def test_maps_refusals(code, changes):
    refused(code, make_maps, **changes)


def test_maps_refuses_overlap_and_a_block_size_without_blocks():
    both = torch.zeros(3, dtype=I32)
    refused(binding.ERR_ALIAS, make_maps, blocks_held=both, blocks_held_out=both)
    head = torch.zeros(1, dtype=I32)
    refused(binding.ERR_ALIAS, make_maps, free_head=head, free_head_out=head)
    none = dict.fromkeys(("block_tables", "blocks_held", "free_blocks", "free_head", "blocks_held_out",
                          "free_head_out", "slot_map"))
    refused(binding.ERR_ARG, make_maps, **none)
    with pytest.raises(ValueError):                        # without blocks at all: every check passes
        fn, args = make_maps()
        fn(**{**args, **none, "block_size": 0})


def test_extra_fields_of_other_calls_are_refused():
    for field, value in (("tile_v", 16), ("schedule", 1), ("reserved", 1), ("workspace_bytes", 8)):
        call = spec.PreparedCommitStates.__new__(spec.PreparedCommitStates)
        fn, args = make_commit()
        call._flags = 0
        with pytest.raises(ValueError):
            call.__init__(**args)
        setattr(call._extra, field, value)
        with pytest.raises(binding.GdnError) as e:
            call._check(call._bind(spec.CHECK_ONLY))
        assert e.value.status == binding.ERR_ARG, field


def test_null_arguments():
    lib = spec.load()
    assert lib.gdn_token_probs(None, None, None, None, 0, None) == binding.ERR_NULL_ARG
    assert lib.gdn_verify_drafts(*[None] * 8, 0, None) == binding.ERR_NULL_ARG
    assert lib.gdn_commit_states(*[None] * 5, 0, None) == binding.ERR_NULL_ARG
    assert lib.gdn_step_maps(None) == binding.ERR_NULL_ARG
    assert lib.gdn_step_maps(ctypes.byref(spec.GdnStepMapsCall())) == binding.ERR_NULL_ARG


def test_plain_forms_by_hand():
    """The 64-bit forms that the GPU tests compare with, on worked cases."""
    p, st = spec_plain.probs(np.array([[0.0, np.log(3.0)], [np.nan, -np.inf], [2.0, 2.0]]), np.array([1.0, 1.0, 0.0]),
                             None, np.zeros((3, 2)))
    assert np.allclose(p, [[0.25, 0.75], [0, 0], [1, 0]]) and st == 0
    # p(x) = 1/2, q(x) = 1: accepted below u = 1/2 only; the residual of a rejection leaves x out
    target = np.array([[0.5, 0.25, 0.25], [0.0, 0.5, 0.5]])
    for u, tokens, n in ((0.49, [0, 1], 2), (0.5, [2, -1], 1)):
        out, num, st = spec_plain.verify(target, np.array([[0]]), None, np.array([[u, 0.5 if n == 1 else 0.25]]),
                                         np.array([0, 2]))
        assert out.tolist() == [tokens] and num.tolist() == [n] and st == 0
    got, st = spec_plain.maps([2, 1], [3, 0], [5, 6], 4, np.array([[7, 0], [0, 0]]), [1, 0], [8, 9], 0, 4)
    assert got["cu_seqlens"].tolist() == [0, 2, 3] and got["positions"].tolist() == [3, 4, 0, -1]
    assert got["slot_map"].tolist() == [31, 32, 36, -1] and got["free_head_out"].tolist() == [2] and st == 0
