// The score kernels' own source (its device part, put in front of this file), one workgroup
// after the other.
extern "C" const char* run_scores(int dtype, int top, int rows, int vocab, int keep, int splits, int per_split,
                                  const int* order, const void* logits, const int32_t* token, const float* temperature,
                                  float* logprob, int32_t* rank, float* entropy, int32_t* top_token, float* top_logprob,
                                  float* norm) {
    using namespace specv;
    const LogprobsArgs a{logits, token, temperature, logprob, rank, entropy, top_token, top_logprob, norm, vocab, keep};
    std::vector<Part> parts(rows * splits);
    std::vector<uint64_t> keys(rows * splits * keep + 1);
    auto main = [&]() {
        auto f = dtype == kBF16 ? top ? logprobs_kernel<kBF16, kT, kU, true> : logprobs_kernel<kBF16, kT, kU, false>
                                : top ? logprobs_kernel<kF32, kT, kU, true> : logprobs_kernel<kF32, kT, kU, false>;
        f(a, splits, per_split, parts.data(), keys.data());
    };
    auto merge = [&]() {
        (dtype == kBF16 ? logprobs_merge_kernel<kBF16> : logprobs_merge_kernel<kF32>)(a, splits, parts.data(), keys.data());
    };
    for (int b = 0; b < rows * splits; ++b)
        if (const char* what = wavefronts::run_group(b, kT, order, main))
            return what;
    for (int b = 0; splits > 1 && b < rows; ++b)
        if (const char* what = wavefronts::run_group(b, kT, order, merge))
            return what;
    return nullptr;
}
