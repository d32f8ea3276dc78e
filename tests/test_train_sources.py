"""Rules of the training operators that their sources show (no GPU)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_moe_ffn_gemv_b200", "csrc")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", text), flags=re.S)


def test_calls_without_a_status_have_no_wait_that_gives_up():
    """The norm calls take no status word, so their kernels hold no wait with a time limit: it
    could only give up in silence."""
    header = open(os.path.join(ROOT, "include", "moe_train.h")).read()
    for call in re.findall(r"moe_norm_\w+\((.*?)\);", header, flags=re.S):
        assert "device_status" not in call
    assert not re.findall(r"\b(mbar_\w+|gtimer|globaltimer|wait_bar|grid_barrier)\b", code("norm.cu"))


def test_no_launch_error_is_dropped():
    """Every launch's status is returned or checked: a failed one between two that work would be
    answered with MOE_OK."""
    for name in sorted(os.listdir(CSRC)):
        if not (name.startswith("train_") or name == "norm.cu") or not name.endswith(".cu"):
            continue
        for line in code(name).splitlines():
            if re.search(r"\blaunch_(chained|spread)\(", line):
                assert re.search(r"return launch_|MOE_LAUNCH\(", line), f"{name}: {line.strip()}"
