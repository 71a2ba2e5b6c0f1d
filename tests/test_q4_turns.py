"""The turns of moe_linear_q4's converter warpgroups, walked through on the host.

A wait for a barrier's phase by its parity also passes while the phase before is still incomplete.  So whoever waits has
to know that one to be complete, from its own earlier waits, whatever the order in which loads land:
- the buffer of step n was free, so step n - A_BUFS and all before it are multiplied;
- a multiplied step's stage of codes, and a stage that the warpgroup saw itself, has come.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
BUFFER, CODES, EXPAND, RELEASE = range(4)
SHAPES = [(32, 0), (64, 0), (128, 0), (64, 1), (64, 3)]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    import __graft_entry__
    b = __graft_entry__._build_module()
    so = str(tmp_path_factory.mktemp("q4_turns") / "q4_turns.so")
    r = subprocess.run([b._nvcc(), *b.ARCH, "-O1", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", f"-I{b.INCLUDE}", "-shared",
                        "-o", so, os.path.join(HERE, "q4_turns.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(so)


def shape_of(lib, columns, parts):
    v = [ctypes.c_int() for _ in range(3)]
    assert lib.q4_shape(columns, parts, *[ctypes.byref(x) for x in v]) == 0
    return [x.value for x in v]


def notes(lib, columns, parts, group, steps, tile, tiles, pairs):
    room = 4 * steps * (-(-(tiles - tile) // pairs)) + 16
    out = np.zeros((room, 4), np.int32)
    n = lib.q4_turns(columns, parts, group, steps, tile, tiles, pairs, out.ctypes.data_as(ctypes.c_void_p), room)
    assert 0 <= n <= room
    return out[:n].tolist()


def stage_of(n, steps):                                        # of all tiles' stages; a tile's last may hold one step
    return n // steps * ((steps + 1) // 2) + n % steps // 2


def first_step(stage, steps):
    per = (steps + 1) // 2
    return stage // per * steps + stage % per * 2


@pytest.mark.parametrize("columns, parts", SHAPES)
def test_every_wait_knows_the_phase_before_to_be_complete(lib, columns, parts):
    converters, buffers, stages = shape_of(lib, columns, parts)
    for steps in range(2, 130):                                # K from 129 on; the kernels begin at 256
        tiles = max(4, 90 // steps)
        for group in range(converters):
            n, known, seen = group, -1, set()                  # turn; last step known to be multiplied; own stages
            for what, slot, parity, _ in notes(lib, columns, parts, group, steps, 0, tiles, 1):
                if what == BUFFER:
                    assert (slot, parity) == (n % buffers, (n // buffers + 1) % 2)
                    assert n - 2 * buffers <= known, (steps, group, n)
                    known = max(known, n - buffers)
                elif what == CODES:
                    q = stage_of(n, steps)
                    assert (slot, parity) == (q % stages, q // stages % 2)
                    before = q - stages
                    assert before < 0 or before in seen or first_step(before, steps) <= known, (steps, group, n)
                    seen.add(q)
                elif what == RELEASE:
                    n += converters
            assert n >= tiles * steps > n - converters


@pytest.mark.parametrize("columns, parts", SHAPES)
def test_every_step_is_expanded_once_and_every_stage_released(lib, columns, parts):
    converters, buffers, stages = shape_of(lib, columns, parts)
    for steps, tile, tiles, pairs in [(2, 0, 5, 1), (3, 1, 9, 4), (4, 0, 3, 76), (7, 2, 230, 76), (23, 75, 400, 76), (16, 3, 2, 5)]:
        mine = len(range(tile, tiles, pairs))
        made, freed = {}, {}
        for group in range(converters):
            n, held = group, []
            for what, slot, a, b in notes(lib, columns, parts, group, steps, tile, tiles, pairs):
                if what == EXPAND:                             # after both waits, on what they were for
                    assert sorted(held) == [(BUFFER, b), (CODES, slot)]
                    assert (slot, a, b) == (stage_of(n, steps) % stages, n % steps % 2, n % buffers) and n not in made
                    made[n] = group
                elif what == RELEASE:
                    q = stage_of(n, steps)
                    assert slot == q % stages
                    freed[q] = freed.get(q, 0) + a
                    n, held = n + converters, []
                else:
                    held.append((what, slot))
        assert sorted(made) == list(range(mine * steps))
        assert set(freed) == set(range(mine * ((steps + 1) // 2))) and all(v == 2 for v in freed.values())


@pytest.mark.parametrize("x_ring", [0, 1])
@pytest.mark.parametrize("columns, parts", SHAPES + [(256, 0)])
def test_no_warpgroup_ends_before_buffers_and_stages_have_been_reported_free(lib, columns, parts, x_ring):
    converters, buffers, _ = shape_of(lib, columns, parts)
    for total in range(2, 300):
        out, rings = np.zeros((32, 3), np.int32), ctypes.c_int()
        n = lib.q4_end(columns, parts, total, x_ring, out.ctypes.data_as(ctypes.c_void_p), ctypes.byref(rings))
        x_stages = rings.value
        assert n == min(total, buffers) + x_ring * min(total, x_stages)
        waits = out[:n].tolist()
        for group in range(converters):
            last = (total - 1 - group) // converters * converters + group          # its last turn, negative if it had none
            known = last - buffers                                                 # multiplied
            for step, (what, slot, parity) in zip(range(total - min(total, buffers), total), waits):
                assert (what, slot, parity) == (0, step % buffers, step // buffers % 2)    # the phase that this step's products end
                assert step < buffers or step - buffers <= known                   # the one before is known to be over
                known = max(known, step)
            assert known == total - 1          # all are: the x of each had come, once its stage's use before was reported
            for step, wait in zip(range(total - min(total, x_stages), total), waits[min(total, buffers):]):
                assert wait == [1, step % x_stages, step // x_stages % 2]


@pytest.mark.parametrize("columns, parts", SHAPES + [(256, 0)])
def test_no_loader_of_codes_ends_before_its_loads_have_landed(lib, columns, parts):
    _, _, stages = shape_of(lib, columns, parts)
    for total in range(1, 200):
        out = np.zeros((stages, 2), np.int32)
        n = lib.q4_codes_end(columns, parts, total, out.ctypes.data_as(ctypes.c_void_p))
        assert n == min(total, stages)
        known = total - 1 - stages                             # the load whose stage was free for the last one
        for load, (slot, parity) in zip(range(total - n, total), out.tolist()):
            assert (slot, parity) == (load % stages, load // stages % 2) and load - stages <= known
