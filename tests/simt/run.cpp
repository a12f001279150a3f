// The order of warps in which the calls that follow run their CTAs, and the errors that they flagged.
extern "C" void simt_order(int order) { simt::order = order; }
extern "C" int simt_parts(int n, int per) { return mla::parts_of(n, per); }
extern "C" int simt_error() {
    const int e = mla_host::error_word;
    mla_host::error_word = 0;
    return e;
}
