"""What a launcher keeps by device from its first call on is published whole: other threads of a program test one
element of it before they read the others, which plain variables do not order (CPU, by reading the sources)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "microscaled_precision_moe_gb300", "csrc")


def test_launchers_keep_atomics_by_device():
    kept = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            source = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\n[ \t]+static\s+(?!constexpr|const\b|cudaError_t|inline)([\w:<> ]+?)[\s*]+(\w+)\s*\[[^;(]*;", source):
            locked = source[m.end():m.end() + 40].lstrip().startswith("static std::mutex")      # or under a mutex
            kept.append((os.path.basename(path), m[2], locked or m[1].startswith("std::atomic<")))
    plain = [k for k in kept if not k[2]]
    assert len(kept) >= 9 and not plain, plain
    # the few-token layer's two numbers: the one that is tested is set last
    with open(os.path.join(CSRC, "moe_few.cu")) as f:
        launch = f.read().split("static cudaError_t launch_few", 1)[1]
    assert launch.index("if (sms[dev] == 0)") < launch.index("fixed[dev] =") < launch.index("sms[dev] = ")
