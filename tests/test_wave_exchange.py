"""Lanes of a wave that hand each other values through LDS (CPU only): a wave barrier orders the
schedule and not memory, so it stands between wavefront-scope fences, in one function."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "allreduce_compatible_gradient_amd", "csrc")


def test_wave_barriers_stand_between_fences():
    uses = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".hip", ".h", ".cpp")):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        uses += text.count("wave_exchange();")
        for m in re.finditer(r"__builtin_amdgcn_wave_barrier\(\);", text):
            before = text[:m.start()].rstrip().splitlines()[-1]
            after = text[m.end():].lstrip().splitlines()[0]
            assert re.search(r'amdgcn_fence\(__ATOMIC_RELEASE, "wavefront"', before), (name, before)
            assert re.search(r'amdgcn_fence\(__ATOMIC_ACQUIRE, "wavefront"', after), (name, after)
    assert uses >= 7
