"""The device error word says what gave up: the tensor-core products' waits share codes 1 to 6,
every other cause has one of its own, which the header names."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "latent_mixture_experts_sigmoid_gb300", "csrc")


def test_codes_are_apart():
    codes = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = open(path).read()
        for name, value in re.findall(r"\b(kErr\w+) = (\d+)", text):
            codes.setdefault(name, {})[os.path.basename(path)] = int(value)
    products = {"grouped.cu", "gemm_tc.cu", "fp8.cu", "fp8_pair.cu", "fp8_stream.cu"}
    own = {}
    for name, where in codes.items():
        for path, value in where.items():
            if path in products:
                assert 1 <= value <= 6, (name, path)
            else:
                assert value > 6 and value not in own, (name, path, value)
                own[value] = name
    header = open(os.path.join(ROOT, "include", "lmoe.h")).read()
    text = header[header.index("Reads (and with clear != 0 resets) the device error word"):header.index("int lmoe_device_error")]
    assert own and all(f"{value} = " in text for value in own), own
